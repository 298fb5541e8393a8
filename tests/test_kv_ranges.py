"""KV cache: lengths past a table row, large scores, values of very different
magnitudes, scales out of range and slots named twice, against the plain forms
of _kv.py."""
import numpy as np
import pytest
import torch

import gguf_quant_dequant_q4_b200 as kq
from tests import _kv
from tests.test_kv_cache import attend, check, flag, i32

pytestmark = pytest.mark.gpu


def rows_of(want, rows):
    """A stand-in for a case whose expected values are some rows of `want`."""
    part = _kv.Case.__new__(_kv.Case)
    part.expected = lambda *a: tuple(x[rows] for x in want)
    return part


# ------------------------------------------------- lengths past the table row
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [4, 12, 60])   # few rows a key head, and prompts
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 20), (False, 0), (False, 20)])
def test_lengths_past_the_table_row(d, new, causal, window):
    # 140 tokens where the row holds 128: positions are those of the given
    # length, and the keys behind the row count as hidden
    case = _kv.Case([(100, 3), (140, new), (0, 0), (139, 1)], 4, 2, d, 16, seed=21)
    want = case.expected(0.1, causal, window, [(1, 8), (3, 8)])
    case.table = np.ascontiguousarray(case.table[:, :8])
    err = flag()
    got = attend(case, 0.1, causal, window, err=err)
    check(rows_of(want, slice(None)), got, 0.1, wide=True)
    assert int(err) == kq.DEV_TOO_MANY
    # an idle request that is too long is nobody's concern
    case.cu = np.array([0, 3, 3, 3, 3], np.int32)
    err.zero_()
    check(rows_of(want, slice(0, 3)), attend(case, 0.1, causal, window, err=err)[:3], 0.1)
    assert int(err) == 0


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 7, 90])
def test_the_longest_length(d, new):
    # positions at the end of 32 bits: every key of the row is visible, none with a window
    case = _kv.Case([(128, new), (50, 1)], 4, 2, d, 16, seed=31, spare=0)
    want = case.expected(0.1, False)
    case.lens[0] = 2 ** 31 - 1
    err = flag()
    check(rows_of(want, slice(None)), attend(case, 0.1, err=err), 0.1, wide=True)
    assert int(err) == kq.DEV_TOO_MANY
    got = attend(case, 0.1, True, 50)
    assert bool((got[:new] == 0).all())
    check(rows_of(want, slice(new, None)), got[new:], 0.1, wide=True)


@pytest.mark.parametrize("d", [64, 192])
@pytest.mark.parametrize("new", [10, 100])
def test_offsets_past_the_tokens(d, new):
    # q holds three tokens less than the offsets say: the others keep their places
    case = _kv.Case([(40, 5), (300, new)], 4, 2, d, 16, seed=22)
    want = case.expected(0.1, True, 50)
    err = flag()
    got = attend(case, 0.1, True, 50, q=case.q[:-3].cuda(), err=err)
    check(rows_of(want, slice(0, 2 + new)), got, 0.1, wide=True)
    assert int(err) == kq.DEV_BAD_RANGE


@pytest.mark.parametrize("hq,d", [(4, 64), (8, 128), (4, 256)])
def test_a_request_that_outgrows_its_row(hq, d):
    """plan, append and attention: 20 cached and 20 new tokens in a row of two
    16-token pages, beside a request that fits."""
    page, hkv, rng = 16, 2, np.random.default_rng(d)
    kp = torch.full((8, hkv, page, d // 32 * 18), 255, dtype=torch.uint8, device="cuda")
    vp = kp.clone()
    free, taken, table, err = i32(rng.permutation(8)), i32([0]), i32(np.full((2, 2), -1)), flag()
    lens = i32([0, 0])
    for step, new in enumerate(([20, 9], [20, 7])):
        lens, cu, slots, pos = kq.kv_plan(lens, i32(new), table, free, taken, page, sum(new), err=err)
        k, v = (torch.from_numpy(rng.standard_normal((sum(new), hkv, d)).astype(np.float32)).cuda() for _ in range(2))
        kq.kv_append(k, v, kp, vp, kq.Q4_0, slots, err=err)
        assert int(err) == (kq.DEV_TOO_MANY if step else 0)
    assert lens.tolist() == [40, 16] and pos[:20].tolist() == list(range(20, 40))
    assert slots[12:20].tolist() == [-1] * 8 and (slots[:12] >= 0).all()
    case = _kv.Case.__new__(_kv.Case)
    case.seqs, case.hq, case.hkv, case.d, case.page = [(40, 20), (16, 7)], hq, hkv, d, page
    tab = table.cpu().numpy()
    case.table = np.concatenate([tab, tab[:, :1]], 1)           # (the third page does not count)
    case.lens, case.cu = np.array([40, 16]), np.array([0, 20, 27])
    case.k, case.v = kp.cpu().numpy(), vp.cpu().numpy()
    case.q = torch.from_numpy(rng.standard_normal((27, hq, d)).astype(np.float32)).to(torch.bfloat16)
    want = case.expected(0.1, True, 0, [(0, 2)])
    err.zero_()
    got = kq.kv_attention(case.q.cuda(), kp, vp, kq.Q4_0, table, lens, cu, 20, scale=0.1, err=err)
    check(rows_of(want, slice(None)), got, 0.1, wide=True)
    assert int(err) == kq.DEV_TOO_MANY


# -------------------------------------------------------- slots named twice
@pytest.mark.parametrize("h,d,t", [(1, 64, 8), (2, 64, 700), (8, 128, 300), (3, 256, 64)])
def test_slots_named_twice(h, d, t):
    # which token's bytes such a slot holds is open, but they are the tokens'
    # own, and every other slot is what it is
    page, rng = 16, np.random.default_rng(t)
    n_pages = 2 * t // page + 2
    slots = rng.permutation(n_pages * page)[:t].astype(np.int32)
    twice = slots[: t // 4].copy()
    slots[t - t // 4:] = twice                     # the last quarter goes where the first went
    k, v = (torch.from_numpy(rng.standard_normal((t, h, d)).astype(np.float32)) for _ in range(2))
    pools = [torch.full((n_pages, h, page, d // 32 * 18), 9, dtype=torch.uint8, device="cuda") for _ in range(2)]
    kq.kv_append(k.cuda(), v.cuda(), pools[0], pools[1], kq.Q4_0, i32(slots))
    for x, pool in ((k, pools[0]), (v, pools[1])):
        rows, got = _kv.encode(x.numpy()), pool.transpose(1, 2).cpu().numpy().reshape(n_pages * page, h, -1)
        once = slots[t // 4:t - t // 4]
        np.testing.assert_array_equal(got[once], rows[t // 4:t - t // 4])
        a, b = rows[: t // 4], rows[t - t // 4:]
        assert ((got[twice] == a) | (got[twice] == b)).all()
        rest = np.setdiff1d(np.arange(n_pages * page), slots)
        assert (got[rest] == 9).all()


# ------------------------------------------------------------- large scores
def steep(seqs, d, q, kdiv):
    """Key j of every sequence is -(j + 1) / kdiv in all of its values and q is
    -1 (even heads) or 1 (odd heads) in all of its: scores are exact, the last
    visible key (or the first) has the largest, by far."""
    case = _kv.Case(seqs, 4, 2, d, 16, seed=23)
    for b, (n, _) in enumerate(seqs):
        for j in range(n):
            case.k[case.table[b, j // 16], :, j % 16] = _kv.encode(np.full((2, d), -(j + 1) / kdiv, np.float32))
    case.q = (torch.tensor([-q, q, -q, q])[:, None] * torch.ones(case.q.shape)).to(torch.bfloat16)
    return case


def check_steep(case, scale):
    # one key has weight 1: P is a power of two, and what is left of check()'s
    # bound are the roundings of P d or a decoded value, and of the output
    want, mag, _, step = case.expected(scale)
    got = attend(case, scale).double().cpu().numpy()
    assert np.isfinite(got).all()
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -10 + 2.0 ** -18) * mag * 1.02 + 2.0 ** -17 * step + 1e-30
    assert (np.abs(got - want) / tol).max() <= 1.0


STEEP = [[(70, 1), (300, 2)], [(200, 3), (33, 16)], [(400, 150), (90, 40)]]


@pytest.mark.parametrize("q", [1e5, 1e6, 1e7, 3e8, 1e9, 1e10, 1e12, 1e20, 1e30])
@pytest.mark.parametrize("seqs", STEEP)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_large_scores(seqs, d, q):
    check_steep(steep(seqs, d, q, 128), d ** -0.5)


@pytest.mark.parametrize("q,scale", [(1e37, 0.0), (1e38, 0.0), (-1e38, 0.0), (3e38, 1e-3), (1e37, -0.05), (1e-38, 1e38), (1e-30, 1e33)])
@pytest.mark.parametrize("seqs", STEEP)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_factors_at_the_ends_of_fp32(seqs, d, q, scale):
    # the scores are finite, while the power of two that brings q to
    # binary16, or its product with the scale, is near fp32's ends
    check_steep(steep(seqs, d, q, 4096), scale or d ** -0.5)


# ---------------------------------------------- values of different magnitudes
def rescale(case, b, j, factor, heads=slice(None), blocks=slice(None)):
    """Multiplies the value scales of token j of sequence b by `factor`."""
    raw = case.v[case.table[b, j // case.page], :, j % case.page].reshape(case.hkv, -1, 18)
    d = np.ascontiguousarray(raw[..., :2]).view(np.float16)[..., 0]
    d[heads, blocks] = (d[heads, blocks].astype(np.float64) * factor).astype(np.float16)
    raw[..., :2] = d[..., None].view(np.uint8)
    case.v[case.table[b, j // case.page], :, j % case.page] = raw.reshape(case.hkv, -1)


SMALL = (-14.0, -12.0)     # exponents of the ordinary value scales


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("seqs,rows", [([(43, 3)], 2), ([(500, 4), (70, 2)], 3), ([(300, 60)], 59)])
def test_a_later_tokens_values_do_not_blur_earlier_rows(d, seqs, rows):
    # the sequence's last token, which only the last row sees, has values 2^24
    # times the others'
    case = _kv.Case(seqs, 4, 2, d, 16, seed=24, v_exp=SMALL)
    rescale(case, 0, seqs[0][0] - 1, 2.0 ** 24)
    got = attend(case, 0.1)
    check(case, got, 0.1, wide=True)
    check(rows_of(case.expected(0.1), slice(0, rows)), got[:rows], 0.1, wide=True)


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("where", [0, 20, 39])
@pytest.mark.parametrize("new", [1, 3, 33])
def test_large_values_of_no_weight(d, where, new):
    # every query is positive and one key is far below zero: its weight is 0,
    # its values 2^24 times the others'
    case = _kv.Case([(40, new)], 4, 2, d, 16, seed=25, v_exp=SMALL)
    case.q = case.q.abs()
    case.k[case.table[0, where // 16], :, where % 16] = _kv.encode(np.full((2, d), -200.0, np.float32))
    rescale(case, 0, where, 2.0 ** 24)
    check(case, attend(case, 0.1), 0.1, wide=True)


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("new", [1, 4, 60])
@pytest.mark.parametrize("low", [-12, -16, -20, -24])
def test_blocks_of_different_magnitudes(d, new, low):
    # the first block's scales are 2^2 and more, the others' 2^low
    case = _kv.Case([(300, new), (70, 1)], 4, 2, d, 16, seed=26, v_exp=(0.0, 1.0))
    for b, (n, _) in enumerate(case.seqs):
        for j in range(n):
            rescale(case, b, j, 4.0, blocks=0)
            rescale(case, b, j, 2.0 ** low, blocks=slice(1, None))
    check(case, attend(case, 0.1), 0.1, wide=True)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 4, 60])
@pytest.mark.parametrize("up", [False, True])
def test_magnitudes_that_rise_or_fall(d, new, up):
    # value scales from 2^12 to 2^-23 along the sequence (or back), and weights
    # that move the other way, by 2^16
    n, hq = 1200, 4
    case = _kv.Case([(n, new)], hq, 2, d, 16, seed=27, v_exp=(0.0, 0.5))
    exps = np.linspace(12, -23, n) if not up else np.linspace(-23, 12, n)
    for j in range(n):
        rescale(case, 0, j, 2.0 ** exps[j])
        case.k[case.table[0, j // 16], :, j % 16] = _kv.encode(np.full((2, d), (-1 if up else 1) * (j - n / 2) / n * 16, np.float32))
    case.q = torch.ones_like(case.q)
    check(case, attend(case, np.log(2) / d), np.log(2) / d, wide=True)


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("fill", [0x3fff, 0x43ff, 0x6fff, 0x0001])
def test_leftovers_in_the_last_page(d, fill):
    # behind the last token lie blocks with finite scales, beside visible ones
    # from 2^12 down to 2^-24
    case = _kv.Case([(37, 2), (70, 3), (5, 1)], 4, 2, d, 16, seed=32, v_exp=(-24.0, 12.0))
    for pool in (case.k, case.v):
        raw = pool.reshape(*pool.shape[:3], -1, 18)
        raw[(raw == 255).all(-1)] = np.frombuffer(np.uint16(fill).tobytes() + bytes([0x1f] * 16), np.uint8)
    for window in (0, 30):
        got = attend(case, 0.02, True, window)
        assert torch.isfinite(got).all()
        check(case, got, 0.02, True, window, wide=True)


# --------------------------------------------------------- scales out of range
@pytest.mark.parametrize("pool", ["k", "v"])
@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("word", [0x7e, 0x7c, 0xfc, 0x71, 0xf1])   # NaN, infinite of both signs, 10240 and more
@pytest.mark.parametrize("new", [1, 6, 50])
def test_scales_out_of_range(pool, d, word, new):
    # the same rule for few rows and for prompts: rows that see the token are
    # not numbers, whatever max_new chooses; the other rows are what they are
    case = _kv.Case([(120, new), (90, 2)], 4, 2, d, 16, seed=28)
    want = case.expected(0.1, True, 4)
    at = max(120 - new - 2, 120 - 30)              # the rows at positions at .. at + 3 see it
    raw = case.k if pool == "k" else case.v
    raw[case.table[0, at // 16], 1, at % 16, 19] = word      # the second block's scale of head 1
    see = np.zeros((new + 2, 4), bool)
    see[:new, 2:] = ((np.arange(120 - new, 120) >= at) & (np.arange(120 - new, 120) < at + 4))[:, None]
    fine = torch.from_numpy(~see)
    for most in (case.max_new, 2000):
        case.max_new = most
        got = attend(case, 0.1, True, 4).cpu()
        assert torch.isnan(got[~fine]).all() and see.any()
        part = rows_of(want, see == False)         # noqa: E712
        check(part, got[fine], 0.1, wide=True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [10, 30])
def test_rows_between_two_scales_out_of_range(d, window):
    # a window that holds neither of the two tokens: the rows between are numbers
    case = _kv.Case([(400, 400), (700, 65)], 2, 1, d, 16, seed=29)
    want = case.expected(0.1, True, window)
    case.k[case.table[0, 130 // 16], 0, 130 % 16, 1] = 0x7e
    case.v[case.table[0, 240 // 16], 0, 240 % 16, 19] = 0x7c
    case.v[case.table[1, 636 // 16], 0, 636 % 16, 19] = 0x7c
    got = attend(case, 0.1, True, window)
    pos = np.concatenate([np.arange(400), 635 + np.arange(65)])
    first = np.arange(465) < 400
    see = np.where(first, ((pos >= 130) & (pos < 130 + window)) | ((pos >= 240) & (pos < 240 + window)),
                   (pos >= 636) & (pos < 636 + window))
    assert torch.isnan(got[torch.from_numpy(see).cuda()]).all()
    fine = np.flatnonzero(~see)
    check(rows_of(want, fine), got[torch.from_numpy(fine).cuda()], 0.1, wide=True)


@pytest.mark.parametrize("d", [64, 128])
def test_many_prompts_beside_scales_out_of_range(d):
    # several short prompts a CTA, some of more than 128 rows a key head; every
    # fifth sequence has a value whose scale is not a number
    rng = np.random.default_rng(d)
    seqs = [(int(n) + 40, int(min(n, m))) for n, m in zip(rng.integers(34, 160, 70), rng.integers(34, 160, 70))]
    case = _kv.Case(seqs, 16, 8, d, 16, seed=30)
    want = case.expected(0.1, True, 40)
    bad = np.zeros((len(case.q), 16), bool)
    for b in range(0, len(seqs), 5):
        n, m = seqs[b]
        at, h = n - m // 2, b % 8
        case.v[case.table[b, at // 16], h, at % 16, 1] = 0x7e
        pos = n - m + np.arange(m)
        bad[case.cu[b]:case.cu[b + 1], 2 * h:2 * h + 2] = ((pos >= at) & (pos < at + 40))[:, None]
    for _ in range(3):
        got = attend(case, 0.1, True, 40).cpu()
        assert torch.isnan(got[torch.from_numpy(bad)]).all()
        check(rows_of(want, ~bad), got[torch.from_numpy(~bad)], 0.1, wide=True)
