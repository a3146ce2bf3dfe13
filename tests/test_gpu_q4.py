"""4-bit pools on the GPU against the fp64 oracle: append, conversion, copies
(bit for bit) and decode attention (element by element).

Tolerance of the attention, from the arithmetic (D dimensions, N tokens):
  out = sum_t w_t v_t.  The output is rounded once (half a step, eps / 2).  Each
  numerator weight, times its scale, is rounded once to fp16: 2^-11 of it, or
  2^-25 of the largest where it is subnormal.  A score is an fp32 sum of D products
  and of the zero point's term, off by at most D 2^-24 scale sum |q| s (n + |z|) =: e;
  (with one or two query heads the products' sums are whole numbers, exact, of queries
  off by at most 2^-22 of the row's largest: for the rows drawn here below e);
  with the exponential's own 2^-22 that moves a weight by a factor of 1 + e + 2^-22,
  in the numerator and in the denominator.  The numerator is an fp32 sum of N
  products, each of which enters a partial sum by rounding or chopping, at most 2^-23 of it:
  off by at most N 2^-23 sum_t w |v|.
"""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_478_b200 as pa
from oracle import compress as oc
from paged_kv_cache_478_b200 import synthetic as syn
from tests.gpu_cases import workspace_for

pytestmark = pytest.mark.gpu

TYPES = {"f16": (torch.float16, pa.PA_Q4_F16), "bf16": (torch.bfloat16, pa.PA_Q4_BF16)}


@pytest.fixture(autouse=True)
def _clean_error_word():
    if torch.cuda.is_available():
        pa.pa_device_errors()
    yield


def as_type(x, kind):
    """numpy -> (CUDA tensor of the type, its exact values as float64)."""
    t = torch.from_numpy(np.ascontiguousarray(x)).to(TYPES[kind][0])
    return t.cuda(), t.double().numpy()


def random_rows(rng, n, heads, dim):
    """Rows whose channels differ in size and offset, with a few outliers."""
    size = np.exp(rng.standard_normal(dim))
    x = rng.standard_normal((n, heads, dim)) * size + 0.5 * size[::-1]
    x[rng.random(x.shape) < 0.01] *= 10
    return x


def filled_pool(rng, nb, heads, dim, kind, fill=0xFF):
    """A pool of quantised random rows, host bytes (fill: other bytes, 0xFF is a NaN scale)."""
    pool = np.full((nb, heads, 9 * dim), fill, dtype=np.uint8)
    _, x = as_type(random_rows(rng, nb * 16, heads, dim), kind)
    for r in range(nb * 16):
        for h in range(heads):
            oc.store_row(pool, r // 16, h, r % 16, x[r, h])
    return pool


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ---- append ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,tokens", [(1, 1), (3, 5), (2, 33), (5, 16)])
def test_append_is_bit_exact(kind, dim, heads, tokens):
    rng = np.random.default_rng(tokens * 10 + heads)
    nb = 4
    kn, kx = as_type(random_rows(rng, tokens, heads, dim), kind)
    vn, vx = as_type(random_rows(rng, tokens, heads, dim), kind)
    slots = rng.permutation(nb * 16)[:tokens].astype(np.int32)
    if tokens > 2:
        slots[1] = -1  # padding
    kp = rng.integers(0, 256, (nb, heads, 9 * dim)).astype(np.uint8)
    vp = rng.integers(0, 256, (nb, heads, 9 * dim)).astype(np.uint8)
    kd, vd = cuda(kp), cuda(vp)
    pool = pa.pa_pool_create(nb, 16, heads, dim, TYPES[kind][1])
    pa.pa_reshape_and_cache(pool, kn, vn, cuda(slots), kd, vd)
    assert pa.pa_device_errors() == 0
    for t in range(tokens):
        for h in range(heads if slots[t] >= 0 else 0):
            oc.store_row(kp, slots[t] // 16, h, slots[t] % 16, kx[t, h])
            oc.store_row(vp, slots[t] // 16, h, slots[t] % 16, vx[t, h])
    assert np.array_equal(kd.cpu().numpy(), kp) and np.array_equal(vd.cpu().numpy(), vp)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_append_of_special_rows(kind):
    """Zeros, constants, far offsets, the type's extremes, subnormals, infinities and NaN."""
    dim, top = 64, float(torch.finfo(TYPES[kind][0]).max)
    tiny = float(torch.finfo(TYPES[kind][0]).smallest_normal) / 8
    rng = np.random.default_rng(3)
    rows = [np.zeros(dim), np.full(dim, 5.0), np.full(dim, -7.25), 1000 + rng.standard_normal(dim),
            np.where(np.arange(dim) % 2, 1.0, -1.0), rng.standard_normal(dim) * tiny,
            np.r_[np.zeros(dim - 1), tiny], np.r_[top, rng.standard_normal(dim - 1)],
            np.r_[np.nan, np.ones(dim - 1)], np.r_[np.ones(dim - 1), np.inf],
            np.r_[-np.inf, np.inf, np.zeros(dim - 2)], np.r_[top, -top, np.zeros(dim - 2)],
            np.arange(dim) / 4.0, -np.arange(dim) / 8.0, np.r_[0.5, 15.5, np.arange(dim - 2) % 16]]
    x = np.stack(rows)[:, None]
    kn, kx = as_type(x, kind)
    pool = pa.pa_pool_create(1, 16, 1, dim, TYPES[kind][1])
    kd, vd = torch.zeros((1, 1, 9 * dim), dtype=torch.uint8, device="cuda"), torch.zeros((1, 1, 9 * dim), dtype=torch.uint8, device="cuda")
    pa.pa_reshape_and_cache(pool, kn, kn, torch.arange(len(rows), dtype=torch.int32, device="cuda"), kd, vd)
    want = np.zeros((1, 1, 9 * dim), dtype=np.uint8)
    for r in range(len(rows)):
        oc.store_row(want, 0, 0, r, kx[r, 0])
    got = oc.values(kd.cpu().numpy(), dim)[0, 0, :len(rows)]
    ref = oc.values(want, dim)[0, 0, :len(rows)]
    assert np.array_equal(got, ref, equal_nan=True)
    assert torch.equal(kd, vd)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_append_of_quotients_at_and_beside_halves(kind):
    """Every scale of 8 bits, near zero and far from it: values at k + 1/2 steps, as near as the
    type holds them, and the type's next numbers above and below."""
    dim, t = 64, TYPES[kind][0]
    step, base = np.meshgrid(np.arange(128, 256) / 64.0, [0.0, -7.0, -8.0, 400.0, -1500.0])
    step, base = step.reshape(-1, 1), base.reshape(-1, 1)
    half = torch.from_numpy(step * (base + np.arange(15) + 0.5)).to(t)
    lo, hi = torch.full_like(half, -float("inf")), torch.full_like(half, float("inf"))
    ends = torch.from_numpy(step * (base + np.array([0.0, 15.0]))).to(t)
    near = [half, torch.nextafter(half, lo), torch.nextafter(half, hi)]
    small = torch.from_numpy(step * (base + np.array([2047.0, 2049.0, 1023.0]) / 4096.0)).to(t)
    x = torch.cat([ends, *near, small], 1)
    x = torch.cat([x, x[:, :dim - x.shape[1]]], 1)[:, None].contiguous()
    n = x.shape[0]
    nb = -(-n // 16)
    pool = pa.pa_pool_create(nb, 16, 1, dim, TYPES[kind][1])
    kd = torch.zeros((nb, 1, 9 * dim), dtype=torch.uint8, device="cuda")
    vd = torch.zeros_like(kd)
    new = x.cuda()
    pa.pa_reshape_and_cache(pool, new, -new, torch.arange(n, dtype=torch.int32, device="cuda"), kd, vd)
    want_k, want_v = np.zeros(kd.shape, dtype=np.uint8), np.zeros(kd.shape, dtype=np.uint8)
    exact = x.double().numpy()
    for r in range(n):
        oc.store_row(want_k, r // 16, 0, r % 16, exact[r, 0])
        oc.store_row(want_v, r // 16, 0, r % 16, -exact[r, 0])
    assert np.array_equal(kd.cpu().numpy(), want_k) and np.array_equal(vd.cpu().numpy(), want_v)


def test_append_reports_bad_slots_and_writes_nothing_there():
    pool = pa.pa_pool_create(2, 16, 3, 64, pa.PA_Q4_F16)
    k = torch.zeros((2, 3, 576), dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    new = torch.ones((2, 3, 64), dtype=torch.float16, device="cuda")
    pa.pa_reshape_and_cache(pool, new, new, torch.tensor([32, -5], dtype=torch.int32, device="cuda"), k, v)
    assert pa.pa_device_errors() == pa.PA_DEVERR_SLOT
    assert not k.any() and not v.any()


# ---- conversion and copies ---------------------------------------------------------------

@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("dim,heads", [(64, 1), (64, 3), (128, 5)])
def test_convert_blocks_both_ways(kind, dim, heads):
    rng = np.random.default_rng(dim + heads)
    nb = 7
    x16, x = as_type(random_rows(rng, nb * 16, heads, dim).reshape(nb, 16, heads, dim).transpose(0, 2, 1, 3), kind)
    y16, y = as_type(random_rows(rng, nb * 16, heads, dim).reshape(nb, 16, heads, dim).transpose(0, 2, 1, 3), kind)
    wide = pa.pa_pool_create(nb, 16, heads, dim, TYPES[kind][0])
    four = pa.pa_pool_create(nb + 2, 16, heads, dim, TYPES[kind][1])
    k4 = torch.zeros((nb + 2, heads, 9 * dim), dtype=torch.uint8, device="cuda")
    v4 = torch.zeros_like(k4)
    pairs = np.array([[0, 8], [6, 1], [2, 2], [3, 0]], dtype=np.int32)
    pa.pa_convert_blocks(wide, x16, y16, four, k4, v4, cuda(pairs))
    assert pa.pa_device_errors() == 0
    want_k, want_v = np.zeros(k4.shape, dtype=np.uint8), np.zeros(k4.shape, dtype=np.uint8)
    for a, b in pairs:
        for h in range(heads):
            for t in range(16):
                oc.store_row(want_k, b, h, t, x[a, h, t])
                oc.store_row(want_v, b, h, t, y[a, h, t])
    assert np.array_equal(k4.cpu().numpy(), want_k) and np.array_equal(v4.cpu().numpy(), want_v)
    back_k, back_v = torch.full_like(x16, 3.0), torch.full_like(x16, 3.0)
    back = np.array([[8, 5], [1, 4], [0, 6]], dtype=np.int32)
    pa.pa_convert_blocks(four, k4, v4, wide, back_k, back_v, cuda(back))
    assert pa.pa_device_errors() == 0
    for got, pool in ((back_k, want_k), (back_v, want_v)):
        ref = torch.full((nb, heads, 16, dim), 3.0, dtype=torch.float64)
        vals = torch.from_numpy(oc.values(pool, dim))
        for a, b in back:
            ref[b] = vals[a]
        assert torch.equal(got.cpu(), ref.to(TYPES[kind][0]))


def test_convert_holds_the_finite_range():
    """fp16: the last step of a group near the type's largest value may pass it."""
    dim = 64
    x = np.zeros((1, 1, 16, dim))
    x[0, 0, :, 0] = 65504.0
    x[0, 0, :, 1] = -np.linspace(1, 65504, 16)
    x16, _ = as_type(x, "f16")
    wide, four = pa.pa_pool_create(1, 16, 1, dim, torch.float16), pa.pa_pool_create(1, 16, 1, dim, pa.PA_Q4_F16)
    k4, v4 = torch.zeros((1, 1, 576), dtype=torch.uint8, device="cuda"), torch.zeros((1, 1, 576), dtype=torch.uint8, device="cuda")
    pairs = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    pa.pa_convert_blocks(wide, x16, x16, four, k4, v4, pairs)
    out = torch.zeros_like(x16)
    pa.pa_convert_blocks(four, k4, v4, wide, out, torch.zeros_like(out), pairs)
    ref = np.clip(oc.values(k4.cpu().numpy(), dim), -65504, 65504)
    assert np.abs(oc.values(k4.cpu().numpy(), dim)).max() > 65504  # the clamp is reached
    assert np.array_equal(out.cpu().double().numpy(), ref.astype(np.float16).astype(np.float64))


def test_convert_and_copy_report_bad_pairs():
    wide, four = pa.pa_pool_create(3, 16, 2, 64, torch.float16), pa.pa_pool_create(5, 16, 2, 64, pa.PA_Q4_F16)
    x = torch.ones((3, 2, 16, 64), dtype=torch.float16, device="cuda")
    k, v = torch.zeros((5, 2, 576), dtype=torch.uint8, device="cuda"), torch.zeros((5, 2, 576), dtype=torch.uint8, device="cuda")
    bad = torch.tensor([[3, 0], [-1, 1], [0, 5], [0, -2], [1, 4]], dtype=torch.int32, device="cuda")
    pa.pa_convert_blocks(wide, x, x, four, k, v, bad)
    assert pa.pa_device_errors() == pa.PA_DEVERR_PAIR
    assert not k[:4].any() and k[4].any()
    pa.pa_copy_blocks(four, k, v, torch.tensor([[4, 0], [5, 1]], dtype=torch.int32, device="cuda"))
    assert pa.pa_device_errors() == pa.PA_DEVERR_PAIR
    assert torch.equal(k[0], k[4]) and torch.equal(v[0], v[4]) and not k[1:4].any()


# ---- decode -------------------------------------------------------------------------------

EDGE_LENGTHS = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 255, 256, 257, 600]


def decode_case(seed, lengths, heads, group, dim, kind, spread=random_rows, shared_rows=None):
    """A decode problem over quantised pools; every byte outside the cached tokens is 0xFF
    (NaN scales), so that anything read there shows."""
    rng = np.random.default_rng(seed)
    need = [-(-n // 16) for n in lengths]
    nb, wide = sum(need) + 1, max(need + [1])
    tables = syn.random_tables(rng, lengths, nb, wide)
    kp = np.full((nb, heads, 9 * dim), 0xFF, dtype=np.uint8)
    vp = kp.copy()
    rows = sum(lengths)
    _, kx = as_type(spread(rng, rows, heads, dim), kind)
    _, vx = as_type(spread(rng, rows, heads, dim), kind)
    r = 0
    for s, n in enumerate(lengths):
        for t in range(n):
            for h in range(heads):
                oc.store_row(kp, tables[s, t // 16], h, t % 16, kx[r, h])
                oc.store_row(vp, tables[s, t // 16], h, t % 16, vx[r, h])
            r += 1
    q, qx = as_type(rng.standard_normal((len(lengths), heads * group, dim)), kind)
    return dict(kp=kp, vp=vp, tables=tables, lens=np.array(lengths, dtype=np.int32), q=q, qx=qx, heads=heads, group=group,
                dim=dim, kind=kind, scale=1 / math.sqrt(dim))


def run_decode(c, partition=0, **kw):
    nb = c["kp"].shape[0]
    pool = pa.pa_pool_create(nb, 16, c["heads"], c["dim"], TYPES[c["kind"]][1])
    pa.pa_pool_set_query_heads(pool, c["heads"] * c["group"])
    out = torch.full_like(c["q"], float("nan"))
    ws = workspace_for(pool, len(c["lens"]), c["tables"].shape[1], 0, partition)
    pa.pa_decode_attention(pool, c["q"], cuda(c["kp"]), cuda(c["vp"]), cuda(c["tables"]), cuda(c["lens"]), c["scale"], out, ws,
                           partition_size=partition, **kw)
    return out


def reference(c):
    n, s, z = oc.parts(c["kp"], c["dim"])
    k, v = oc.values(c["kp"], c["dim"]), oc.values(c["vp"], c["dim"])
    out, weights, bound = oc.attend(c["qx"], k, v, c["lens"], c["tables"], c["scale"])
    eps = torch.finfo(TYPES[c["kind"]][0]).eps
    tol = np.zeros_like(out)
    mag = np.repeat(s, 64, -1) * (n + np.abs(np.repeat(z, 64, -1)))
    for i, L in enumerate(c["lens"]):
        for h in range(out.shape[1] if L else 0):
            hk = h // c["group"]
            rows = np.stack([mag[c["tables"][i, t // 16], hk, t % 16] for t in range(L)])
            vals = np.stack([v[c["tables"][i, t // 16], hk, t % 16] for t in range(L)])
            e = c["dim"] * 2.0 ** -24 * c["scale"] * (rows @ np.abs(c["qx"][i, h])).max() + 2.0 ** -22
            tol[i, h] = (eps / 2 * np.abs(out[i, h]) * 1.01 + (1.01 * 2.0 ** -11 + 2 * e) * bound[i, h]
                         + L * 2.0 ** -23 * bound[i, h] + L * 2.0 ** -25 * np.abs(vals).max() + torch.finfo(TYPES[c["kind"]][0]).smallest_normal * eps)
    return out, tol, weights


def check(got, want, tol):
    g = got.double().cpu().numpy()
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.nanmax(np.abs(g - want) / np.maximum(tol, 1e-30))))


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,group", [(1, 1), (2, 4), (3, 2), (6, 1), (1, 8), (4, 8)])
def test_decode_lengths_and_heads(kind, dim, heads, group):
    lengths = EDGE_LENGTHS if heads * group <= 8 else [0, 1, 17, 64, 130, 257]
    c = decode_case(heads * 100 + group, lengths, heads, group, dim, kind)
    want, tol, _ = reference(c)
    for partition in (0, 16, 64, 208):
        check(run_decode(c, partition), want, tol)
        assert pa.pa_device_errors() == 0


def offset_rows(rng, n, heads, dim):
    return 50 + rng.standard_normal((n, heads, dim))


def sized_rows(rng, n, heads, dim):
    """Tokens whose sizes differ by many powers of two."""
    return rng.standard_normal((n, heads, dim)) * 2.0 ** rng.integers(-12, 3, (n, 1, 1))


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("spread", [offset_rows, sized_rows])
def test_decode_of_uneven_values(kind, spread):
    c = decode_case(5, [200, 77, 16], 2, 4, 128, kind, spread)
    want, tol, _ = reference(c)
    for partition in (0, 64):
        check(run_decode(c, partition), want, tol)


def test_decode_of_large_and_small_bf16_values():
    """Values far outside fp16's range, in a type that holds them."""
    for size in (1e30, 1e-30):
        c = decode_case(6, [100, 3], 1, 2, 64, "bf16", lambda rng, n, h, d: size * rng.standard_normal((n, h, d)))
        c["q"], c["qx"] = as_type(c["qx"] / size, "bf16")
        want, tol, _ = reference(c)
        check(run_decode(c), want, tol)


def test_nan_values_reach_their_own_group_only():
    c = decode_case(7, [40], 1, 1, 128, "f16")
    row = oc.values(c["vp"], 128)[c["tables"][0, 1], 0, 3].copy()
    row[100] = np.nan
    oc.store_row(c["vp"], c["tables"][0, 1], 0, 3, row)
    got = run_decode(c)[0, 0]
    assert torch.isnan(got[64:]).all() and torch.isfinite(got[:64]).all()


@pytest.mark.parametrize("scale", [0.0, -0.125])
def test_zero_and_negative_scales(scale):
    c = dict(decode_case(13, [100, 17, 64], 2, 2, 64, "f16"), scale=scale)
    want, _, _ = reference(c)
    _, tol, _ = reference(dict(c, scale=abs(scale)))  # the same magnitudes
    bound = oc.attend(c["qx"], oc.values(c["kp"], 64), oc.values(c["vp"], 64), c["lens"], c["tables"], scale)[2]
    check(run_decode(c), want, np.maximum(tol, 2.0 ** -10 * bound + 2.0 ** -20))


def test_a_nan_key_reaches_its_own_head_only():
    c = decode_case(14, [70], 2, 1, 64, "bf16")
    row = oc.values(c["kp"], 64)[c["tables"][0, 2], 1, 9].copy()
    row[5] = np.inf
    oc.store_row(c["kp"], c["tables"][0, 2], 1, 9, row)
    for partition in (0, 16):
        got = run_decode(c, partition)[0]
        assert torch.isnan(got[1]).all() and torch.isfinite(got[0]).all()


def test_bad_block_ids_are_reported():
    c = decode_case(8, [40, 20], 2, 1, 64, "f16")
    c["tables"][0, 1] = 10 ** 6
    c["tables"][1, 0] = -3
    run_decode(c)
    assert pa.pa_device_errors() == pa.PA_DEVERR_BLOCK_ID


def test_results_repeat_bit_for_bit_and_do_not_depend_on_placement():
    c = decode_case(9, [300, 50], 2, 2, 128, "bf16")
    a = run_decode(c, 64)
    assert torch.equal(a, run_decode(c, 64))
    nb = c["kp"].shape[0]
    perm = np.random.default_rng(1).permutation(nb)
    moved = dict(c, kp=c["kp"][np.argsort(perm)], vp=c["vp"][np.argsort(perm)],
                 tables=np.where(c["tables"] >= 0, perm[c["tables"]], -1).astype(np.int32))
    assert torch.equal(a, run_decode(moved, 64))


@pytest.mark.parametrize("group", [1, 4])
def test_append_and_attend_planned_in_a_graph(group):
    """The serving step: plan once, then append + attend, captured on a side stream and
    replayed; the same as the separate calls, pools included."""
    lengths = [1, 16, 17, 0, 140]
    c = decode_case(10, lengths, 3, group, 128, "f16")
    S, heads, dim = len(lengths), 3, 128
    rng = np.random.default_rng(4)
    kn, vn = as_type(random_rows(rng, S, heads, dim), "f16")[0], as_type(random_rows(rng, S, heads, dim), "f16")[0]
    nb = c["kp"].shape[0]
    pool = pa.pa_pool_create(nb, 16, heads, dim, pa.PA_Q4_F16)
    pa.pa_pool_set_query_heads(pool, heads * group)
    bt, cl = cuda(c["tables"]), cuda(c["lens"])
    k1, v1, k2, v2 = (cuda(x) for x in (c["kp"], c["vp"], c["kp"], c["vp"]))
    ws1, ws2 = (workspace_for(pool, S, bt.shape[1], 0, 64) for _ in range(2))
    slots = cuda(pa.pa_decode_slots(c["tables"], c["lens"]))
    want, got, once = (torch.full_like(c["q"], float("nan")) for _ in range(3))
    pa.pa_reshape_and_cache(pool, kn, vn, slots, k1, v1)
    pa.pa_decode_attention(pool, c["q"], k1, v1, bt, cl, c["scale"], want, ws1, partition_size=64)
    k3, v3 = cuda(c["kp"]), cuda(c["vp"])
    pa.pa_decode_append_attention(pool, c["q"], kn, vn, k3, v3, bt, cl, c["scale"], once, ws1, partition_size=64)
    assert torch.equal(once, want) and torch.equal(k3, k1) and torch.equal(v3, v1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pa.pa_decode_plan(pool, cl, bt.shape[1], ws2, partition_size=64)
        pa.pa_decode_append_attention_planned(pool, c["q"], kn, vn, k2, v2, bt, c["scale"], got, ws2, partition_size=64)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(k2, k1) and torch.equal(v2, v1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        pa.pa_decode_append_attention_planned(pool, c["q"], kn, vn, k2, v2, bt, c["scale"], got, ws2, partition_size=64)
    for _ in range(3):
        got.fill_(float("nan"))
        k2.copy_(cuda(c["kp"]))
        v2.copy_(cuda(c["vp"]))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(k2, k1) and torch.equal(v2, v1)
    assert pa.pa_device_errors() == 0


def test_planned_calls_refuse_a_plan_of_another_pool_type():
    c = decode_case(11, [20], 4, 1, 64, "f16")
    nb = c["kp"].shape[0]
    wide, four = pa.pa_pool_create(nb, 16, 4, 64, torch.float16), pa.pa_pool_create(nb, 16, 4, 64, pa.PA_Q4_F16)
    ws = workspace_for(four, 1, c["tables"].shape[1])
    pa.pa_decode_plan(wide, cuda(c["lens"]), c["tables"].shape[1], ws)
    with pytest.raises(pa.PagedAttnError) as e:
        pa.pa_decode_attention_planned(four, c["q"], cuda(c["kp"]), cuda(c["vp"]), cuda(c["tables"]), c["scale"],
                                       torch.empty_like(c["q"]), ws)
    assert e.value.status == 1


def test_static_scratch():
    c = decode_case(12, [100, 31], 2, 2, 64, "bf16")
    nb = c["kp"].shape[0]
    pool = pa.pa_pool_create(nb, 16, 2, 64, pa.PA_Q4_BF16)
    pa.pa_pool_set_query_heads(pool, 4)
    out = torch.empty_like(c["q"])
    pa.pa_decode_attention_static(pool, c["q"], cuda(c["kp"]), cuda(c["vp"]), cuda(c["tables"]), cuda(c["lens"]), c["scale"], out,
                                  partition_size=64)
    assert torch.equal(out, run_decode(c, 64))


def test_wrong_tensors_are_refused_by_the_binding():
    pool = pa.pa_pool_create(2, 16, 2, 64, pa.PA_Q4_F16)
    k = torch.zeros((2, 2, 576), dtype=torch.uint8, device="cuda")
    new = torch.ones((1, 2, 64), dtype=torch.float16, device="cuda")
    slot = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        pa.pa_reshape_and_cache(pool, new, new, slot, k[:1], k)
    with pytest.raises(TypeError):
        pa.pa_reshape_and_cache(pool, new, new, slot, k.view(torch.int8), k)
    with pytest.raises(TypeError):
        pa.pa_reshape_and_cache(pool, new.bfloat16(), new, slot, k, k)


def test_two_streams_at_once():
    """Two decode calls in flight together, each with its own workspace and output."""
    cases = [decode_case(15, [300, 40], 4, 2, 128, "f16"), decode_case(16, [90, 500, 1], 2, 8, 64, "bf16")]
    want = [run_decode(c, 64) for c in cases]
    streams, got, keep = [torch.cuda.Stream() for _ in cases], [], []
    for c, st in zip(cases, streams):
        pool = pa.pa_pool_set_query_heads(pa.pa_pool_create(c["kp"].shape[0], 16, c["heads"], c["dim"], TYPES[c["kind"]][1]), c["heads"] * c["group"])
        args = [cuda(c[k]) for k in ("kp", "vp", "tables", "lens")]
        keep.append((pool, args, workspace_for(pool, len(c["lens"]), c["tables"].shape[1], 0, 64), torch.empty_like(c["q"])))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, st, (pool, (k, v, bt, cl), ws, out) in zip(cases, streams, keep):
            pa.pa_decode_attention(pool, c["q"], k, v, bt, cl, c["scale"], out, ws, partition_size=64, stream=st)
    torch.cuda.synchronize()
    for (_, _, _, out), w in zip(keep, want):
        assert torch.equal(out, w)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes: append, attention, copy and conversion in its last blocks
    give what they give in a small pool."""
    heads, dim, nb = 32, 128, 120000
    assert nb * heads * 9 * dim > 2 ** 32
    c = decode_case(17, [70, 33], heads, 1, dim, "f16")
    want = run_decode(c)
    small = c["kp"].shape[0]
    k = torch.zeros((nb, heads, 9 * dim), dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    k[-small:], v[-small:] = cuda(c["kp"]), cuda(c["vp"])
    far = dict(c, tables=np.where(c["tables"] >= 0, c["tables"] + nb - small, -1).astype(np.int32))
    pool = pa.pa_pool_create(nb, 16, heads, dim, pa.PA_Q4_F16)
    out = torch.empty_like(c["q"])
    ws = workspace_for(pool, 2, c["tables"].shape[1])
    pa.pa_decode_attention(pool, c["q"], k, v, cuda(far["tables"]), cuda(c["lens"]), c["scale"], out, ws)
    assert torch.equal(out, want)
    wide = pa.pa_pool_create(2, 16, heads, dim, torch.float16)
    x = torch.randn((2, heads, 16, dim), dtype=torch.float16, device="cuda")
    back = torch.zeros_like(x)
    pa.pa_convert_blocks(wide, x, x, pool, k, v, torch.tensor([[0, nb - 1], [1, 3]], dtype=torch.int32, device="cuda"))
    pa.pa_convert_blocks(pool, k, v, wide, back, torch.zeros_like(x), torch.tensor([[nb - 1, 1], [3, 0]], dtype=torch.int32, device="cuda"))
    assert (back.flip(0) - x).abs().max() <= 0.5  # a step of N(0, 1) rows is about 0.3
    pa.pa_copy_blocks(pool, k, v, torch.tensor([[nb - 1, nb - 2]], dtype=torch.int32, device="cuda"))
    assert torch.equal(k[nb - 2], k[nb - 1]) and k[nb - 1].any()
    new = x[0, :, :1].permute(1, 0, 2).contiguous()
    pa.pa_reshape_and_cache(pool, new, new, torch.tensor([(nb - 2) * 16 + 5], dtype=torch.int32, device="cuda"), k, v)
    row = oc.values(k[nb - 2:nb - 1].cpu().numpy(), dim)[0, :, 5]
    assert np.abs(row - new[0].double().cpu().numpy()).max() <= 0.5
    assert pa.pa_device_errors() == 0


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_append_far_from_zero(kind):
    """Groups whose offset is many times their range: quotients up to 2000, halves among them."""
    rng = np.random.default_rng(18)
    T, dim = 512, 64
    x = rng.integers(-2000, 2000, (T, 1, 1)) * 0.5 + rng.integers(0, 64, (T, 1, dim)) * 0.25
    kn, kx = as_type(x, kind)
    vn, vx = as_type(x[::-1] * 2.0 ** rng.integers(-10, 3, (T, 1, 1)), kind)
    pool = pa.pa_pool_create(T // 16, 16, 1, dim, TYPES[kind][1])
    kd, vd = torch.zeros((T // 16, 1, 9 * dim), dtype=torch.uint8, device="cuda"), torch.zeros((T // 16, 1, 9 * dim), dtype=torch.uint8, device="cuda")
    pa.pa_reshape_and_cache(pool, kn, vn, torch.arange(T, dtype=torch.int32, device="cuda"), kd, vd)
    kp, vp = np.zeros(kd.shape, dtype=np.uint8), np.zeros(kd.shape, dtype=np.uint8)
    for t in range(T):
        oc.store_row(kp, t // 16, 0, t % 16, kx[t, 0])
        oc.store_row(vp, t // 16, 0, t % 16, vx[t, 0])
    assert np.array_equal(kd.cpu().numpy(), kp) and np.array_equal(vd.cpu().numpy(), vp)
