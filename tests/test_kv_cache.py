"""KV cache in q4_0 pages: plan, append and attention, against the plain forms
of _kv.py (loops and float64 over the CPU oracle's decode)."""
import ctypes

import numpy as np
import pytest
import torch

import gguf_quant_dequant_q4_b200 as kq
import oracle
from tests import _kv

OK, INVALID, UNSUPPORTED, ALIGN = 0, 1, 2, 3
A, MIS = 0x10000, 0x10008   # fake device addresses, never dereferenced
gpu = pytest.mark.gpu


def i32(a):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32).cuda()


def flag():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------ refusals (CPU)
def test_plan_refusals():
    f = kq.lib().kq_kv_plan

    def call(n=2, page=16, table=A, blocks=4, free=A, n_free=8, taken=A, out=A, cu=A, slots=A, cap=8, cached=A, seq=A):
        return f(cached, A, n, page, table, blocks, free, n_free, taken, out, seq, cu, A, slots, None, cap, None, None)

    assert call(n=-1) == INVALID
    assert call(n=2**20 + 1) == INVALID
    for page in (0, -16, 8, 24, 65552):
        assert call(page=page) == UNSUPPORTED
    assert call(blocks=-1) == INVALID
    assert call(blocks=2**30) == INVALID            # blocks * page past 2^30
    assert call(blocks=2**62) == INVALID            # no overflow of the product
    assert call(n_free=-1) == INVALID
    assert call(cap=-1) == INVALID
    assert call(cap=2**30 + 1) == INVALID
    for name in ("table", "free", "taken", "out", "cu", "slots", "cached", "seq"):
        assert call(**{name: None}) == INVALID, name


def test_append_refusals():
    f = kq.lib().kq_kv_append

    def call(qt=kq.Q4_0, k=A, v=A, ty=30, t=2, ks=512, vs=512, h=4, d=128, slots=A, kp=A, vp=A, pages=4, page=16):
        return f(qt, k, v, ty, t, ks, vs, h, d, slots, kp, vp, pages, page, None, None)

    assert call(qt=kq.Q8_0) == UNSUPPORTED
    assert call(ty=1) == UNSUPPORTED
    for d in (0, 32, 96, 80, 320):
        assert call(d=d, ks=4096, vs=4096) == UNSUPPORTED
    assert call(h=0) == INVALID
    assert call(t=-1) == INVALID
    assert call(t=2**30 + 1) == INVALID
    assert call(ks=511) == INVALID                  # tokens would overlap
    assert call(vs=504) == INVALID
    assert call(ks=516) == ALIGN                    # 16-byte rows
    assert call(ty=0, ks=514) == ALIGN
    assert call(page=20) == UNSUPPORTED
    assert call(pages=2**31) == INVALID
    assert call(pages=2**27, page=16) == INVALID    # slots past 32 bits
    for name in ("k", "v", "slots", "kp", "vp"):
        assert call(**{name: None}) == INVALID, name
    for name in ("k", "v", "kp", "vp"):
        assert call(**{name: MIS}) == ALIGN, name
    assert call(t=0) == OK


def test_attention_refusals():
    f = kq.lib().kq_kv_attention

    def call(qt=kq.Q4_0, q=A, t=2, qs=1024, hq=8, h=4, d=128, cu=A, lens=A, n=2, most=1, kp=A, vp=A, pages=4, page=16, tab=A,
             blocks=4, scale=1.0, window=0, out=A, ws=A, wb=1 << 40):
        return f(qt, q, t, qs, hq, h, d, cu, lens, n, most, kp, vp, pages, page, tab, blocks, scale, 1, window, out, ws, wb,
                 None, None)

    assert call(qt=kq.Q4_K) == UNSUPPORTED
    assert call(hq=6, h=4) == INVALID               # heads not a multiple of the key heads
    assert call(hq=2, h=4) == INVALID
    assert call(h=0) == INVALID
    for d in (32, 96, 288):
        assert call(d=d, qs=8192) == UNSUPPORTED
    assert call(qs=1016) == INVALID
    assert call(qs=1028) == ALIGN
    assert call(most=0) == INVALID
    assert call(window=-1) == INVALID
    assert call(scale=float("nan")) == INVALID
    assert call(scale=float("inf")) == INVALID
    assert call(scale=3e38) == INVALID               # (infinite as a base-2 scale)
    assert call(page=8) == UNSUPPORTED
    assert call(blocks=2**40) == INVALID
    assert call(t=2**30 + 1) == INVALID
    assert call(wb=16) == INVALID                   # work space too small
    for name in ("q", "cu", "lens", "kp", "vp", "tab", "out", "ws"):
        assert call(**{name: None}) == INVALID, name
    for name in ("q", "kp", "vp", "out", "ws"):
        assert call(**{name: MIS}) == ALIGN, name
    assert call(t=0) == OK
    assert call(n=0) == OK
    b = ctypes.c_int64()
    w = kq.lib().kq_kv_attention_workspace
    assert w(8, 4, 128, 1, ctypes.byref(b)) == OK and b.value > 0
    assert w(8, 3, 128, 1, ctypes.byref(b)) == INVALID
    assert w(8, 4, 100, 1, ctypes.byref(b)) == UNSUPPORTED
    assert w(8, 4, 128, 0, ctypes.byref(b)) == INVALID
    assert w(8, 4, 128, 1, None) == INVALID


def test_workspace_never_shrinks_with_max_new():
    for hq, h, d in ((8, 8, 64), (32, 4, 128), (24, 3, 192), (16, 2, 256)):
        got = [kq.kv_attention_workspace(hq, h, d, m) for m in (1, 2, 3, 4, 8, 16, 17, 64, 1000, 100000)]
        assert got == sorted(got)


def test_binding_checks():
    cuda = "CUDA tensors"
    z = dict(dtype=torch.int32)
    lens, table, free = torch.zeros(3, **z), torch.zeros(3, 5, **z), torch.zeros(9, **z)
    one = torch.zeros(1, **z)
    with pytest.raises(ValueError, match=cuda):
        kq.kv_plan(lens, lens, table, free, one, 16, 8)
    with pytest.raises(ValueError, match=r"\[3, max_blocks\]"):
        kq.kv_plan(lens, lens, table[:2], free, one, 16, 8)
    with pytest.raises(ValueError, match="at least 3 elements"):
        kq.kv_plan(lens, lens[:2], table, free, one, 16, 8)
    with pytest.raises(TypeError, match="4-byte elements"):
        kq.kv_plan(lens.long(), lens, table, free, one, 16, 8)
    with pytest.raises(ValueError, match="contiguous"):
        kq.kv_plan(lens, lens, torch.zeros(5, 3, **z).t(), free, one, 16, 8)
    row = kq.row_bytes(kq.Q4_0, 64)
    pool = torch.zeros(2, 4, 16, row, dtype=torch.uint8)
    k = torch.zeros(3, 4, 64)
    with pytest.raises(ValueError, match=cuda):
        kq.kv_append(k, k, pool, pool, kq.Q4_0, lens)
    fused = torch.zeros(3, 12 * 64)
    with pytest.raises(ValueError, match=cuda):     # a view of a wider product's columns
        kq.kv_append(fused[:, 256:512].unflatten(1, (4, 64)), fused[:, 512:].unflatten(1, (4, 64)), pool, pool, kq.Q4_0, lens)
    with pytest.raises(ValueError, match="must be contiguous"):
        kq.kv_append(k.transpose(1, 2).contiguous().transpose(1, 2), k, pool, pool, kq.Q4_0, lens)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        kq.kv_append(k.half(), k.half(), pool, pool, kq.Q4_0, lens)
    with pytest.raises(ValueError, match="one shape and type"):
        kq.kv_append(k, k.bfloat16(), pool, pool, kq.Q4_0, lens)
    with pytest.raises(ValueError, match="rows of 36 bytes"):
        kq.kv_append(k, k, torch.zeros(2, 4, 16, 72, dtype=torch.uint8), pool, kq.Q4_0, lens)
    with pytest.raises(ValueError, match=r"\[pages, 4,"):
        kq.kv_append(k, k, pool[:, :2], pool, kq.Q4_0, lens)
    with pytest.raises(ValueError, match="at least 3 elements"):
        kq.kv_append(k, k, pool, pool, kq.Q4_0, lens[:2])
    q, cu = torch.zeros(3, 8, 64, dtype=torch.bfloat16), torch.zeros(4, **z)
    with pytest.raises(ValueError, match=cuda):
        kq.kv_attention(q, pool, pool, kq.Q4_0, table, lens, cu, 1)
    with pytest.raises(TypeError, match="bfloat16"):
        kq.kv_attention(q.float(), pool, pool, kq.Q4_0, table, lens, cu, 1)
    with pytest.raises(ValueError, match="at least 4 elements"):
        kq.kv_attention(q, pool, pool, kq.Q4_0, table, lens, cu[:3], 1)
    with pytest.raises(ValueError, match="at least 1536 elements"):
        kq.kv_attention(q, pool, pool, kq.Q4_0, table, lens, cu, 1, out=q[:2])
    with pytest.raises(ValueError, match=r"\[3, max_blocks\]"):
        kq.kv_attention(q, pool, pool, kq.Q4_0, table[:1], lens, cu, 1)


# -------------------------------------------------------------------- plan
def run_plan(cached, new, page, seed=0, extra=5, taken=3, spare=2, in_place=False):
    rng = np.random.default_rng(seed)
    cached, new = np.asarray(cached, np.int32), np.asarray(new, np.int32)
    held = -(-cached // page)
    most = int((-(-(cached + new) // page)).max(initial=0)) + spare
    need = int((-(-(cached + new) // page) - held).sum())
    perm = rng.permutation(int(held.sum()) + need + taken + 4).astype(np.int32)
    table = np.full((len(cached), most), -7, np.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = perm[at:at + n]
        at += n
    free = perm[at:]
    cap = int(new.sum()) + extra
    want = _kv.plan(cached.tolist(), new.tolist(), table, free, taken, page, cap)
    tab, tk, err = i32(table), i32([taken]), flag()
    out = None if in_place else i32([-1])
    seq, cu, slots, pos = kq.kv_plan(i32(cached), i32(new), tab, i32(free), tk, page, cap, taken_out=out, err=err)
    got = (seq, cu, slots, pos, tab)
    for g, w, what in zip(got, want, ("seq_lens", "cu_new", "slots", "positions", "table")):
        np.testing.assert_array_equal(g.cpu().numpy(), w, err_msg=what)
    assert int((tk if in_place else out)[0]) == want[5]
    assert int(err) == 0


@gpu
@pytest.mark.parametrize("cached,new,page", [
    ([0], [1], 16), ([15, 16, 17, 31], [1, 1, 1, 1], 16), ([0, 0, 0], [0, 0, 0], 16), ([5], [0], 32),
    ([0, 100, 7, 0, 64], [0, 33, 0, 129, 64], 64), ([47, 48, 49], [48, 0, 200], 48), ([0], [9000], 16),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan(cached, new, page, in_place):
    run_plan(cached, new, page, in_place=in_place)


@gpu
@pytest.mark.parametrize("n,top,page", [(31, 3, 16), (1025, 2, 32), (2500, 9, 16), (700, 60, 128)])
def test_plan_many(n, top, page):
    rng = np.random.default_rng(n)
    run_plan(rng.integers(0, 300, n), rng.integers(0, top, n), page, extra=0 if n == 31 else 700)


@gpu
def test_plan_of_no_requests():
    seq, cu, slots, pos = kq.kv_plan(i32([]), i32([]), i32(np.zeros((0, 4))), i32([1, 2]), i32([1]), 16, 5,
                                     taken_out=(out := i32([0])))
    assert seq.numel() == 0 and cu.tolist() == [0] and slots.tolist() == [-1] * 5 and pos.tolist() == [-1] * 5
    assert out.tolist() == [1]


@gpu
@pytest.mark.parametrize("cap", [24, 5000])   # one launch, two launches
def test_plan_lengths_in_place_and_flags(cap):
    # seq_lens may be cached_lens in the C ABI
    cached, new = i32([3, 20]), i32([5, 10])
    table = i32([[4, -1], [9, 2]])
    first, cu, slots, free, taken = i32([0, 0]), i32([0] * 3), i32([7] * cap), i32([11, 12]), i32([0])
    err = flag()

    def call(n_free=2, cap_=cap):
        return kq.lib().kq_kv_plan(cached.data_ptr(), new.data_ptr(), 2, 16, table.data_ptr(), 2, free.data_ptr(), n_free,
                                   taken.data_ptr(), taken.data_ptr(), cached.data_ptr(), cu.data_ptr(), first.data_ptr(),
                                   slots.data_ptr(), None, cap_, err.data_ptr(), torch.cuda.current_stream().cuda_stream)

    assert call() == OK
    assert cached.tolist() == [8, 30] and cu.tolist() == [0, 5, 15] and taken.tolist() == [0] and int(err) == 0
    assert slots[:15].tolist() == [4 * 16 + p for p in range(3, 8)] + [2 * 16 + p for p in range(4, 14)]
    assert set(slots[15:].tolist()) == {-1}
    # the second request runs past its table row; the first takes one of two pages
    assert call() == OK
    assert cached.tolist() == [13, 40] and int(err) == kq.DEV_TOO_MANY and table.tolist() == [[4, -1], [9, 2]]
    assert slots[5:15].tolist() == [2 * 16 + 14, 2 * 16 + 15] + [-1] * 8
    err.zero_()
    cached.copy_(i32([13, 0]))
    table.fill_(-1)
    table[0, 0] = 4
    assert call(n_free=1) == OK                  # 13 + 5 and 0 + 10 need two pages, one is left
    assert int(err) == kq.DEV_TOO_MANY and taken.tolist() == [1] and table.tolist() == [[4, 11], [-1, -1]]
    assert slots[:15].tolist() == [4 * 16 + 13, 4 * 16 + 14, 4 * 16 + 15, 11 * 16, 11 * 16 + 1] + [-1] * 10


@gpu
def test_plan_cuts_at_cap_and_bad_lengths():
    err = flag()
    table = i32(np.full((4, 3), -1))
    seq, cu, slots, pos = kq.kv_plan(i32([0, 0, 0, 0]), i32([4, 2**31 - 1, 2**31 - 1, 3]), table, i32([5, 6, 7]), i32([0]), 16,
                                     20, err=err)
    assert int(err) == kq.DEV_TOO_MANY
    assert seq.tolist() == [4, 16, 0, 0] and cu.tolist() == [0, 4, 20, 20, 20]
    assert slots.tolist() == [80, 81, 82, 83] + list(range(96, 112))
    err.zero_()
    table.fill_(0)
    seq, cu, slots, pos = kq.kv_plan(i32([-5, 1000, 2, 48]), i32([2, 1, -1, 0]), table, i32([5, 6]), i32([-1]), 16, 4, err=err)
    assert int(err) == kq.DEV_BAD_RANGE | kq.DEV_TOO_MANY
    assert seq.tolist() == [2, 49, 2, 48] and cu.tolist() == [0, 2, 3, 3, 3]
    assert slots.tolist() == [80, 81, -1, -1] and pos.tolist() == [0, 1, 48, -1]
    err.zero_()
    table.fill_(-1)                              # a held page that is none
    _, _, slots, _ = kq.kv_plan(i32([5, 0, 0, 0]), i32([1, 0, 0, 0]), table, i32([5]), i32([0]), 16, 1, err=err)
    assert slots.tolist() == [-1] and int(err) == kq.DEV_BAD_RANGE


# ------------------------------------------------------------------ append
def append_values(rng, t, h, d, f32):
    x = rng.standard_normal((t, h, d)).astype(np.float32) * 2.0 ** rng.integers(-12, 8, (t, h, 1))
    x = x.reshape(t, h, d // 32, 32)
    x[rng.random(x.shape[:-1]) < 0.05] = 0                       # blocks of zeros
    flat = x.reshape(-1, 32)
    flat[::7, 5] = -np.abs(flat[::7]).max(-1)                    # equal magnitudes of both signs
    flat[::7, 20] = np.abs(flat[::7]).max(-1)
    flat[3::11] = np.float32(2.0 ** -24) * rng.integers(-3, 4, flat[3::11].shape)   # scales that round to zero, or nearly
    x = x.reshape(t, h, d).astype(np.float32)
    return torch.from_numpy(x) if f32 else torch.from_numpy(x).to(torch.bfloat16)


@gpu
@pytest.mark.parametrize("t,h,d,page", [(1, 1, 64, 16), (5, 3, 128, 48), (77, 8, 128, 16), (33, 5, 192, 32), (130, 2, 256, 64),
                                        (1000, 7, 64, 128)])
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("fused", [False, True])
def test_append(t, h, d, page, f32, fused):
    rng = np.random.default_rng(t + d)
    k, v = append_values(rng, t, h, d, f32), append_values(rng, t, h, d, f32)
    n_pages = -(-t // page) + 3
    slots = rng.permutation(n_pages * page)[:t].astype(np.int32)
    if t > 1:
        slots[t // 2::9] = -1
    row = d // 32 * 18
    before = [rng.integers(0, 256, (n_pages, h, page, row), dtype=np.uint8) for _ in range(2)]
    pools = [torch.from_numpy(b.copy()).cuda() for b in before]
    kd, vd = k.cuda(), v.cuda()
    if fused:
        both = torch.full((t, 3 * h * d), 7.0, dtype=k.dtype, device="cuda")
        both[:, h * d:2 * h * d], both[:, 2 * h * d:] = kd.flatten(1), vd.flatten(1)
        kd, vd = both[:, h * d:2 * h * d].unflatten(1, (h, d)), both[:, 2 * h * d:].unflatten(1, (h, d))
    err = flag()
    kq.kv_append(kd, vd, pools[0], pools[1], kq.Q4_0, i32(slots), err=err)
    assert int(err) == 0
    for x, b, got in ((k, before[0], pools[0]), (v, before[1], pools[1])):
        rows = _kv.encode(x.float().numpy())
        for i, s in enumerate(slots):
            if s >= 0:
                b[s // page, :, s % page] = rows[i]
        np.testing.assert_array_equal(got.cpu().numpy(), b)
    # the pool reads back through the library's own decode
    back = kq.dequantize(pools[0], kq.Q4_0, d).cpu().numpy()
    i = int(np.flatnonzero(slots >= 0)[0])
    np.testing.assert_array_equal(back[slots[i] // page, :, slots[i] % page], oracle.dequantize(kq.Q4_0, _kv.encode(k[i].float().numpy()), d))


@gpu
def test_append_round_trip_bound():
    # d = m / 8 and codes 0..15 around 8: off by at most half a step, a whole
    # one at the end that code 16 would take, and d's own rounding (8 * 2^-11)
    x = torch.randn(64, 4, 128, generator=torch.Generator().manual_seed(1))
    pool = torch.zeros(4, 4, 16, 72, dtype=torch.uint8, device="cuda")
    kq.kv_append(x.cuda(), x.cuda(), pool, pool.clone(), kq.Q4_0, i32(np.arange(64)))
    back = kq.dequantize(pool, kq.Q4_0, 128).cpu().transpose(1, 2).reshape(64, 4, 128)
    step = x.reshape(64, 4, 4, 32).abs().amax(-1, keepdim=True) / 8
    assert bool(((back - x).reshape(64, 4, 4, 32).abs() <= step * (1 + 8 * 2.0 ** -11 + 2.0 ** -20)).all())


@gpu
def test_append_flags():
    row = kq.row_bytes(kq.Q4_0, 64)
    pool = torch.full((2, 2, 16, row), 3, dtype=torch.uint8, device="cuda")
    kp, vp = pool.clone(), pool.clone()
    x = torch.ones(4, 2, 64, device="cuda")
    err = flag()
    kq.kv_append(x, x, kp, vp, kq.Q4_0, i32([-1, 32, -2, 2**31 - 1]), err=err)
    assert int(err) == kq.DEV_BAD_RANGE
    assert torch.equal(kp, pool) and torch.equal(vp, pool)
    for bad in (float("inf"), float("-inf"), float("nan"), 3e38):
        err.zero_()
        y = x.clone()
        y[1, 1, 40] = bad
        kq.kv_append(x, y, kp, vp, kq.Q4_0, i32([0, 1, 2, 3]), err=err)
        assert int(err) == kq.DEV_X_RANGE, bad
        got = kq.dequantize(vp, kq.Q4_0, 64)[0, :, :4]
        fine = torch.ones(2, 4, 64, dtype=torch.bool, device="cuda")
        fine[1, 1, 32:] = False
        assert torch.equal(got[fine], torch.ones_like(got[fine])) and not torch.isfinite(got[1, 1, 40])
    err.zero_()
    y = x.clone()
    y[2, 0, 3] = -65504.0                        # the largest magnitude that is not flagged
    kq.kv_append(x, y, kp, vp, kq.Q4_0, i32([0, 1, 2, 3]), err=err)
    assert int(err) == 0
    y[2, 0, 3] = 66000.0
    kq.kv_append(x, y, kp, vp, kq.Q4_0, i32([0, 1, 2, 3]), err=err)
    assert int(err) == kq.DEV_X_RANGE and float(kq.dequantize(vp, kq.Q4_0, 64)[0, 0, 2, 3]) > 57000
    err.zero_()
    y = x.clone()
    y[1, 1, 40] = float("nan")                   # not flagged where nothing is stored
    kq.kv_append(y, y, kp, vp, kq.Q4_0, i32([0, -1, 2, 3]), err=err)
    assert int(err) == 0


# --------------------------------------------------------------- attention
# Bounds.  Output: half a bf16 step, 2^-8 |o|.  P and P * d are rounded to
# binary16 (2^-11 each); where the tensor cores take whole values instead of
# codes, P, k and v are (2^-11 each), a rounded k moving a score by at most
# 2^-11 scale sum |q k|.  Either way at most 2 * 2^-11 of sum p |v|, plus the
# scores' error twice (numerator and sum).  fp32 score sums: up to 288 terms of
# codes below 16 times q, against 8 after the offset: 23 / 8 of sum |q k| at
# most where |k| is at its largest, so 2^-13 scale sum |q k| is generous for the
# rest (exp2, sums, rescaling, joins: 2^-18).  Where an element's values are 0
# (code 8) next to a large block scale, sum p |v| is small and one more error
# counts: fp32 sums hold code * (P d) and -8 * (P d), which cancel.  The sums
# are at most 15 sum p |d| < 2 * step (step = sum p 8 |d|), an MMA adds at most
# 2^-22 of what it holds, and a warp's share of these cases is at most 16
# tiles of 32 keys, 4 MMAs each: 64 * 2^-22 * 2 step = 2^-15 step, on paper;
# the rounding errors' mean is zero, so 2^-17 step is taken.
def check(case, got, scale, causal=True, window=0, hidden=(), wide=False):
    want, mag, big, step = case.expected(scale, causal, window, hidden)
    t = want.shape[0]
    got = got[:t].double().cpu().numpy()
    assert np.isfinite(got).all()
    ey = (2.0 ** -11 if wide else 0.0) * big + 2.0 ** -13 * big
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -10 + 2.0 ** -18 + 2.02 * ey) * mag * 1.02 + 2.0 ** -17 * step + 1e-30
    worst = (np.abs(got - want) / tol).max() if t else 0.0
    assert worst <= 1.0, f"error / bound = {worst:.3f}"
    return worst


def attend(case, scale, causal=True, window=0, out=None, err=None, q=None, **kw):
    return kq.kv_attention(case.q.cuda() if q is None else q, torch.from_numpy(case.k).cuda(), torch.from_numpy(case.v).cuda(),
                           kq.Q4_0, i32(case.table), i32(case.lens), i32(case.cu), case.max_new, scale=scale, causal=causal,
                           window=window, out=out, err=err, **kw)


LENS = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 255, 256, 257, 511]


@gpu
@pytest.mark.parametrize("hq,hkv,d,page", [
    (8, 8, 64, 16), (6, 2, 64, 32), (28, 4, 128, 16), (32, 4, 128, 64), (16, 1, 128, 48), (5, 1, 192, 16), (12, 4, 192, 128),
    (4, 2, 256, 32), (24, 2, 256, 16), (40, 2, 64, 16),
])
def test_one_token(hq, hkv, d, page):
    case = _kv.Case([(n, 1) for n in LENS], hq, hkv, d, page, seed=d + hq)
    err = flag()
    check(case, attend(case, d ** -0.5, err=err), d ** -0.5)
    assert int(err) == 0


@gpu
@pytest.mark.parametrize("seqs,hq,hkv,d", [
    ([(1, 1)], 1, 1, 64), ([(5000, 1)], 8, 2, 128), ([(20011, 1), (3, 1)], 4, 1, 64), ([(7777, 1)], 16, 1, 256),
    ([(300, 1), (0, 0), (0, 0), (9000, 1), (1, 1), (0, 0)], 8, 4, 128), ([(4097, 1)] * 3, 3, 3, 192),
])
def test_one_token_long_and_idle(seqs, hq, hkv, d):
    case = _kv.Case(seqs, hq, hkv, d, 16, seed=len(seqs))
    check(case, attend(case, 0.1), 0.1)


@gpu
@pytest.mark.parametrize("seqs", [[(3, 3), (40, 5), (33, 1), (200, 4)], [(1, 1), (17, 2), (500, 8)]])
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (6, 2, 128), (16, 2, 128), (4, 1, 192), (8, 2, 256)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 7), (True, 64), (False, 0), (False, 20)])
def test_few_tokens(seqs, hq, hkv, d, causal, window):
    case = _kv.Case(seqs, hq, hkv, d, 16, seed=7)
    check(case, attend(case, d ** -0.5, causal, window), d ** -0.5, causal, window, wide=True)


@gpu
@pytest.mark.parametrize("seqs", [[(300, 300)], [(200, 129), (77, 77), (40, 1), (0, 0), (513, 500), (33, 3)], [(2500, 70)],
                                  [(1, 1), (700, 257), (128, 128), (1000, 33)], [(5000, 65), (64, 64), (129, 129)]])
@pytest.mark.parametrize("hq,hkv,d,page", [(4, 4, 64, 16), (3, 1, 64, 48), (8, 2, 128, 32), (7, 1, 128, 16), (16, 1, 128, 64)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 100), (False, 0)])
def test_prompts(seqs, hq, hkv, d, page, causal, window):
    case = _kv.Case(seqs, hq, hkv, d, page, seed=11)
    err = flag()
    check(case, attend(case, d ** -0.5, causal, window, err=err), d ** -0.5, causal, window, wide=True)
    assert int(err) == 0


@gpu
@pytest.mark.parametrize("hq,hkv,d", [(6, 2, 192), (8, 2, 256)])
def test_prompts_of_wide_heads(hq, hkv, d):
    case = _kv.Case([(150, 150), (300, 40), (17, 1)], hq, hkv, d, 32, seed=12)
    check(case, attend(case, d ** -0.5, True, 50), d ** -0.5, True, 50)


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_rows_that_see_nothing_bad_pages_and_padding(d):
    # more new tokens than keys, no keys at all, hidden pages, rows of no sequence
    case = _kv.Case([(200, 200), (0, 40), (300, 150), (5, 1)], 4, 2, d, 16, seed=13, pad=5)
    case.lens[0] = 90                              # its first 110 tokens are before key 0
    hidden = [(2, 0), (2, 9), (2, 18)]
    want = case.expected(0.2, True, 0, hidden)
    for i, (b, j) in enumerate(hidden):
        case.table[b, j] = (-1, case.n_pages, 2**31 - 1)[i]
    out = torch.full((case.q.shape[0], 4, d), 5.0, dtype=torch.bfloat16, device="cuda")
    err = flag()
    got = attend(case, 0.2, out=out, err=err)
    assert int(err) == kq.DEV_BAD_RANGE
    case.expected = lambda *a: want
    check(case, got, 0.2, hidden=hidden, wide=True)
    assert bool((got[:110] == 0).all()) and bool((got[200:240] == 0).all()) and bool((got[391:] == 5).all())


@gpu
@pytest.mark.parametrize("k_exp,v_exp,q_scale,scale", [
    ((-4, -1), (-23, -20), 1.0, 0.1), ((-4, -1), (9, 12.5), 1.0, 0.1), ((-20, -18), (-4, 0), 1e5, 0.5),
    ((8, 10), (-4, 0), 1e-6, 10.0), ((-4, -1), (-4, 0), 1e30, 1e-30), ((-4, -1), (-4, 0), 1.0, 0.0),
    ((-4, -1), (-4, 0), 1.0, -0.2), ((-2, 0), (-4, 0), 8.0, 1.0),
])
def test_prompt_ranges(k_exp, v_exp, q_scale, scale):
    case = _kv.Case([(333, 200), (600, 65)], 4, 2, 128, 16, seed=14, k_exp=k_exp, v_exp=v_exp, q_scale=q_scale)
    check(case, attend(case, scale), scale, wide=True)


@gpu
@pytest.mark.parametrize("slope", [0.08, 0.4, 3.0])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("seqs", [[(700, 300), (300, 140)], [(900, 1), (130, 2)]])
def test_scores_that_rise_or_fall(seqs, d, slope):
    # every key's score is `slope` above (even heads) or below (odd heads) the
    # one before: the reference moves with every few keys, or never
    case = _kv.Case(seqs, 4, 2, d, 16, seed=15)
    for b, (n, _) in enumerate(seqs):
        for j in range(n):
            case.k[case.table[b, j // 16], :, j % 16] = _kv.encode(np.full((2, d), -j / 128, np.float32))
    case.q = (torch.tensor([-1.0, 1.0, -1.0, 1.0])[:, None] * torch.ones_like(case.q)).to(torch.bfloat16)
    scale = slope * 128 / d
    check(case, attend(case, scale), scale, wide=True)


@gpu
def test_rows_that_see_nothing_and_rows_of_no_sequence():
    # a sequence without keys, and one with more new tokens than keys: zeros;
    # the padded rows behind the last sequence stay as they were
    case = _kv.Case([(0, 2), (40, 1), (3, 3)], 4, 2, 64, 16, pad=3)
    case.lens[2] = 1                               # its first two tokens are before key 0
    out = torch.full((9, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    got = attend(case, 0.2, out=out)
    assert got is out
    check(case, got, 0.2)
    assert bool((got[:2] == 0).all()) and bool((got[3:5] == 0).all()) and bool((got[5] != 0).any())
    assert bool((got[6:] == 5).all())


@gpu
@pytest.mark.parametrize("window", [1, 16, 33, 1000])
def test_window_does_not_read_dropped_pages(window):
    # pages wholly before every window are given up (-1, or another's page of NaN)
    case = _kv.Case([(300, 1), (77, 2), (16, 1)], 8, 2, 128, 16, seed=3)
    want = case.expected(0.1, True, window)
    kept = case.table.copy()
    for b, (n, m) in enumerate(case.seqs):
        gone = max(0, n - m - window + 1) // 16
        case.table[b, :gone] = np.where(np.arange(gone) % 2 == 0, -1, case.n_pages + 9)
    err = flag()
    got = attend(case, 0.1, True, window, err=err)
    assert int(err) == 0
    case.table = kept
    case.expected = lambda *a: want
    check(case, got, 0.1, True, window)


@gpu
def test_bad_pages_are_flagged_and_hidden():
    case = _kv.Case([(100, 1), (64, 2), (20, 1)], 4, 2, 64, 16, seed=5)
    hidden = [(0, 2), (1, 0), (1, 3), (2, 0), (2, 1)]
    want = case.expected(0.3, True, 0, hidden)
    for i, (b, j) in enumerate(hidden):
        case.table[b, j] = (-1, case.n_pages, 2**31 - 1, -2**31, case.n_pages + 5)[i]
    err = flag()
    got = attend(case, 0.3, err=err)
    assert int(err) == kq.DEV_BAD_RANGE
    case.expected = lambda *a: want
    check(case, got, 0.3, hidden=hidden, wide=True)
    assert bool((got[3] == 0).all())               # every page of the last sequence


@gpu
@pytest.mark.parametrize("k_exp,v_exp,q_scale,scale", [
    ((-4, -1), (-23, -20), 1.0, 0.1), ((-4, -1), (9, 12.5), 1.0, 0.1), ((-4, -1), (-20, 8), 1.0, 0.1),
    ((-20, -18), (-4, 0), 1e5, 0.5), ((8, 10), (-4, 0), 1e-6, 10.0), ((-4, -1), (-4, 0), 1e30, 1e-30),
    ((-4, -1), (-4, 0), 1.0, 0.0), ((-4, -1), (-4, 0), 1.0, -0.2), ((-2, 0), (-4, 0), 8.0, 1.0),
])
def test_ranges(k_exp, v_exp, q_scale, scale):
    case = _kv.Case([(333, 1), (50, 2), (2000, 1)], 8, 2, 128, 16, seed=9, k_exp=k_exp, v_exp=v_exp, q_scale=q_scale)
    check(case, attend(case, scale), scale, wide=True)


@gpu
def test_values_that_are_not_numbers_stay_with_their_rows():
    # a non-finite value scale reaches only the rows that see the token
    case = _kv.Case([(40, 4)], 4, 2, 64, 16, seed=2)
    want = case.expected(0.1)
    case.v[case.table[0, 2], :, 7, 1] = 0x7e       # token 39 (the last): NaN scale of its first block
    got = attend(case, 0.1)
    assert not torch.isfinite(got[3, :, :32]).any()
    case.expected = lambda *a: tuple(x[:3] for x in want)
    check(case, got, 0.1, wide=True)
    # a query that is not a number: flagged, its row is not a number, the others are
    case = _kv.Case([(40, 2)], 4, 2, 64, 16, seed=2)
    q = case.q.clone()
    q[0, 1, 3] = float("nan")
    err = flag()
    got = attend(case, 0.1, q=q.cuda(), err=err)
    assert int(err) == kq.DEV_X_RANGE and torch.isnan(got[0, 1]).all()
    fine = torch.ones(2, 4, dtype=torch.bool)
    fine[0, 1] = False
    assert torch.isfinite(got[fine.cuda()]).all()


@gpu
@pytest.mark.parametrize("pool", ["k", "v"])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_keys_whose_scale_is_not_finite(pool, d):
    # token 100 of 200: the rows that see it are not numbers, the others are
    # what they are, on either side of it (a window of 30)
    case = _kv.Case([(200, 200), (150, 90)], 2, 1, d, 16, seed=6)
    want = case.expected(0.1, True, 30)
    raw = case.k if pool == "k" else case.v
    at = case.table[0, 100 // 16], 0, 100 % 16
    for word in (0x7e, 0x7c, 0x71):                # NaN, infinite, 10240 and more
        raw[at][19] = word
        got = attend(case, 0.1, True, 30)
        assert not torch.isfinite(got[100:130]).any()
        fine = [i for i in range(290) if not 100 <= i < 130]
        part = _kv.Case.__new__(_kv.Case)
        part.expected = lambda *a: tuple(x[fine] for x in want)
        check(part, got[fine], 0.1, wide=True)


@gpu
@pytest.mark.parametrize("seqs", [[(70, 1), (300, 1)], [(70, 3), (300, 40)], [(400, 150)]])
def test_strided_q_workspace_and_streams(seqs):
    case = _kv.Case(seqs, 6, 2, 128, 32, seed=4)
    t = case.q.shape[0]
    plain = attend(case, 0.1)
    wide = torch.full((t, 10 * 128), 9.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 256:1024] = case.q.flatten(1).cuda()
    q = wide[:, 256:1024].unflatten(1, (6, 128))
    assert torch.equal(attend(case, 0.1, q=q), plain)
    ws = torch.full((kq.kv_attention_workspace(6, 2, 128, case.max_new) + 512,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(attend(case, 0.1, workspace=ws), plain)
    with pytest.raises(kq.KQError, match="invalid argument"):
        attend(case, 0.1, workspace=ws[:16])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    args = (q, torch.from_numpy(case.k).cuda(), torch.from_numpy(case.v).cuda(), kq.Q4_0, i32(case.table), i32(case.lens),
            i32(case.cu), case.max_new)
    torch.cuda.synchronize()
    got = [kq.kv_attention(*args, scale=0.1, stream=s) for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(g, plain) for g in got)
    # a larger bound on the new tokens changes kernels, not meaning
    check(case, kq.kv_attention(*args[:-1], 4000, scale=0.1), 0.1, wide=True)


# ------------------------------------------------------------------ together
@gpu
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (8, 8, 128)])
def test_prompts_then_tokens(hq, hkv, d):
    """Ragged prompts, then single tokens, then a few tokens, with one request
    idle in between: every step's output against the whole history in float64."""
    page, n_pages, rng = 16, 64, np.random.default_rng(d)
    row = d // 32 * 18
    kp = torch.full((n_pages, hkv, page, row), 255, dtype=torch.uint8, device="cuda")
    vp = kp.clone()
    free = i32(rng.permutation(n_pages))
    taken, lens, table = i32([0]), i32([0, 0, 0]), i32(np.full((3, 20), -1))
    err = flag()
    for step, new in enumerate(([37, 1, 150], [1, 1, 1], [1, 0, 1], [4, 17, 0], [1, 1, 1])):
        t = sum(new)
        lens, cu, slots, pos = kq.kv_plan(lens, i32(new), table, free, taken, page, t + 2, err=err)
        qkv = torch.from_numpy(rng.standard_normal((t + 2, (hq + 2 * hkv) * d)).astype(np.float32)).cuda()
        k, v = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)), qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        kq.kv_append(k, v, kp, vp, kq.Q4_0, slots, err=err)
        q = qkv[:, :hq * d].to(torch.bfloat16).unflatten(1, (hq, d))
        got = kq.kv_attention(q, kp, vp, kq.Q4_0, table, lens, cu, max(new), err=err)
        assert int(err) == 0
        case = _kv.Case.__new__(_kv.Case)
        case.seqs, case.hq, case.hkv, case.d, case.page = list(zip(lens.tolist(), new)), hq, hkv, d, page
        case.table, case.lens, case.cu = table.cpu().numpy(), lens.cpu().numpy(), cu.cpu().numpy()
        case.k, case.v, case.q = kp.cpu().numpy(), vp.cpu().numpy(), q.cpu()
        assert case.cu.tolist() == [0] + np.cumsum(new).tolist()
        check(case, got, d ** -0.5, wide=True)
    assert int(taken[0]) == sum(_kv.pages(n, page) for n in lens.tolist())


@gpu
def test_captured_step_replays_with_other_lengths():
    """plan, append and attention of a decode step in one graph: replays follow
    the lengths, tables and inputs that the device memory holds then."""
    hq, hkv, d, page = 8, 2, 128, 16
    rng = np.random.default_rng(8)
    kp = torch.full((40, hkv, page, 72), 255, dtype=torch.uint8, device="cuda")
    vp = kp.clone()
    free, table = i32(rng.permutation(40)), i32(np.full((2, 12), -1))
    taken, lens, one = i32([0]), i32([0, 0]), i32([1, 1])
    kv = torch.empty(2, 2 * hkv * d, device="cuda")
    q = torch.empty(2, hq, d, dtype=torch.bfloat16, device="cuda")

    def step():
        seq, cu, slots, _ = kq.kv_plan(lens, one, table, free, taken, page, 2)
        lens.copy_(seq)
        k, v = kv[:, :hkv * d].unflatten(1, (hkv, d)), kv[:, hkv * d:].unflatten(1, (hkv, d))
        kq.kv_append(k, v, kp, vp, kq.Q4_0, slots)
        return kq.kv_attention(q, kp, vp, kq.Q4_0, table, lens, cu, 1)

    def inputs():
        kv.copy_(torch.from_numpy(rng.standard_normal((2, 2 * hkv * d)).astype(np.float32)))
        q.copy_(torch.from_numpy(rng.standard_normal((2, hq, d)).astype(np.float32)))

    inputs()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    # a second graph with its own work space, replayed on another stream in between
    other = _kv.Case([(777, 1), (9, 1)], hq, hkv, d, page, seed=1)
    oargs = (other.q.cuda(), torch.from_numpy(other.k).cuda(), torch.from_numpy(other.v).cuda(), kq.Q4_0, i32(other.table),
             i32(other.lens), i32(other.cu), 1)
    kq.kv_attention(*oargs)
    g2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g2):
        out2 = kq.kv_attention(*oargs)
    torch.cuda.synchronize()
    for i in range(40):
        inputs()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g2.replay()
        g.replay()
        torch.cuda.synchronize()
        if i in (0, 14, 15, 16, 31, 39):
            case = _kv.Case.__new__(_kv.Case)
            case.seqs, case.hq, case.hkv, case.d, case.page = [(int(n), 1) for n in lens], hq, hkv, d, page
            case.table, case.lens, case.cu = table.cpu().numpy(), lens.cpu().numpy(), np.array([0, 1, 2])
            case.k, case.v, case.q = kp.cpu().numpy(), vp.cpu().numpy(), q.cpu()
            check(case, out, d ** -0.5)
            check(other, out2, d ** -0.5)
    assert lens.tolist() == [41, 41]               # one call outside the graph, 40 replays
