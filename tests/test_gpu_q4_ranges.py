"""Decode over 4-bit pools whose keys and values differ in size by many powers of two, on
the GPU against the fp64 oracle: the softmax sum must not depend on the values, nor small
values of the attended tokens on large ones of tokens that are not attended.

Tolerance, from the arithmetic (L tokens, D dimensions, w the normalised weights, s a group's
scale, n - z a held value; every bound is for one dimension of one head):
  * the output's own rounding, eps / 2 of it (and half a subnormal step);
  * scores: fp32 sums, off by at most D 2^-24 scale sum |q| s (n + |z|) + 2^-22 =: e, numerator
    and denominator: 2 e sum w |v|;
  * P = w s 2^k held as two fp16 numbers: 2^-21 of it, and where they are subnormal 2^-25.  2^k puts the
    largest w s so far at 2^10 or above (2^3 at least where k meets its limit of 126: scales down
    to 2^-123): a subnormal is off by 2^-28 of the largest, times |n - z|;
  * the sum of the numerator: L 2^-23 sum w |v|;
  * weights below 2^-126 of the largest are zero: L 2^-125 max |v|;
  * partial results: the running maximum plus a whole number, below 2^7, is off by 2^-18, a
    weight of a partition by as much: 2^-17 sum w |v|.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_478_b200 as pa
from oracle import compress as oc
from tests.test_gpu_q4 import TYPES, as_type, check, cuda, decode_case, run_decode

pytestmark = pytest.mark.gpu

ROUNDED = 2.0 ** -21  # of a weight times its scale


@pytest.fixture(autouse=True)
def _clean_error_word():
    if torch.cuda.is_available():
        pa.pa_device_errors()
    yield


def sized(k_size, v_size):
    """Rows N(0, 1) times a size per token (and dimension): K first, then V, as decode_case draws them."""
    sizes = [np.asarray(k_size, dtype=np.float64), np.asarray(v_size, dtype=np.float64)]

    def spread(rng, n, heads, dim):
        size = sizes.pop(0)
        size = np.broadcast_to(size.reshape(-1, 1, size.shape[1] if size.ndim == 2 else 1), (n, 1, size.shape[1] if size.ndim == 2 else 1))
        return rng.standard_normal((n, heads, dim)) * size

    return spread


def expected(c):
    """Output, its tolerance and the weights of a decode_case."""
    dim, (ns, ss, zs) = c["dim"], oc.parts(c["vp"], c["dim"])
    kn, ks, kz = oc.parts(c["kp"], dim)
    kmag = np.repeat(ks, 64, -1) * (kn + np.abs(np.repeat(kz, 64, -1)))
    held = np.abs(ns - np.repeat(zs, 64, -1))
    v = oc.values(c["vp"], dim)
    out, weights, bound = oc.attend(c["qx"], oc.values(c["kp"], dim), v, c["lens"], c["tables"], c["scale"])
    fi = torch.finfo(TYPES[c["kind"]][0])
    tol, rel = np.zeros_like(out), [np.zeros(out.shape[1]) for _ in c["lens"]]
    for i, L in enumerate(c["lens"]):
        b, r = c["tables"][i, np.arange(L) // 16], np.arange(L) % 16
        for h in range(out.shape[1] if L else 0):
            hk, w = h // c["group"], weights[i][h]
            e = dim * 2.0 ** -24 * abs(c["scale"]) * (kmag[b, hk, r] @ np.abs(c["qx"][i, h])).max() + 2.0 ** -22
            largest = np.repeat((w[:, None] * ss[b, hk, r]).max(0), 64) * np.repeat(held[b, hk, r].reshape(L, -1, 64).max((0, 2)), 64)
            tol[i, h] = (fi.eps / 2 * 1.01 * np.abs(out[i, h]) + fi.smallest_normal * fi.eps / 2
                         + (ROUNDED * 1.01 + 2.02 * e + L * 2.0 ** -23 + 2.0 ** -17) * bound[i, h]
                         + L * 2.0 ** -28 * largest + L * 2.0 ** -125 * np.abs(v[b, hk, r]).max(0))
            rel[i][h] = 2 * e + 2.0 ** -17
    return out, tol, weights, rel


def check_decode_and_mass(c, partitions=(0, 16, 64, 208)):
    want, tol, weights, rel = expected(c)
    S, HQ = want.shape[:2]
    pool = pa.pa_pool_set_query_heads(pa.pa_pool_create(c["kp"].shape[0], 16, c["heads"], c["dim"], TYPES[c["kind"]][1]), HQ)
    k, v, bt, cl = (cuda(c[n]) for n in ("kp", "vp", "tables", "lens"))
    for partition in partitions:
        got = run_decode(c, partition)
        check(got, want, tol)
        ws = torch.empty(pa.pa_decode_mass_workspace_bytes(pool, S, bt.shape[1], 0, partition), dtype=torch.uint8, device="cuda")
        out, mass = torch.empty_like(c["q"]), torch.zeros((S, bt.shape[1] * 16), device="cuda")
        pa.pa_decode_attention_mass(pool, c["q"], k, v, bt, cl, c["scale"], out, None, mass, ws, partition_size=partition)
        assert pa.pa_device_errors() == 0 and torch.equal(out, got)
        for i, L in enumerate(c["lens"]):
            # the weights, which know nothing of V: a factor of 1 + rel each, (HQ + 2) 2^-24 for their sum
            off = np.abs(mass[i, :L].double().cpu().numpy() - weights[i].sum(0))
            assert (off <= (rel[i][:, None] * weights[i]).sum(0) + (HQ + 2) * 2.0 ** -24 * weights[i].sum(0) + HQ * 2.0 ** -125).all()


# ---- values of every size, comparable scores -------------------------------------------------

SIZES = {"zeros_then_1e14": lambda t: np.where(t < 64, 0, 1e14), "1e14_then_zeros": lambda t: np.where(t < 64, 1e14, 0),
         "tiny_then_huge": lambda t: np.where(t < 64, 1e-30, 1e30), "huge_then_tiny": lambda t: np.where(t < 64, 1e30, 1e-30),
         "rising": lambda t: 10.0 ** (t / 5 - 36), "falling": lambda t: 10.0 ** (36 - t / 5), "mixed": lambda t: 10.0 ** (t * 7919 % 73 - 36),
         "zeros_amid_huge": lambda t: np.where(t % 3, 0, 1e37)}


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("heads,group,dim", [(1, 1, 64), (6, 1, 128), (2, 2, 128), (1, 4, 64), (4, 4, 128), (2, 8, 128)])
def test_values_of_very_different_sizes(sizes, heads, group, dim):
    lengths = [360, 129, 1] if heads * group <= 8 else [300]
    t = np.concatenate([np.arange(n) for n in lengths])
    c = decode_case(heads + group + dim, lengths, heads, group, dim, "bf16", sized(np.full(len(t), 0.5), SIZES[sizes](t)))
    check_decode_and_mass(c)


# ---- large values that are not attended --------------------------------------------------------

def shunned(kind, group, dim, at, big, small, away, heads=1, turned=False):
    """`small` values everywhere but at the tokens `at`, whose values are `big` and whose scores lie `away` (natural
    units) below the others.  turned: the group's last query head attends to those instead."""
    L = 330
    c = decode_case(7 * group + dim, [L], heads, group, dim, kind, sized(np.full(L, 0.02), np.where(np.isin(np.arange(L), at), big, small)))
    base = np.random.default_rng(5).standard_normal(dim)
    qx = base + 0.05 * np.random.default_rng(6).standard_normal((1, heads * group, dim))
    if turned:
        qx[:, group - 1::group] *= -1
    c["q"], c["qx"] = as_type(qx, kind)
    row = -away / (c["scale"] * (base @ base)) * base
    for t in at:
        for h in range(heads):
            oc.store_row(c["kp"], c["tables"][0, t // 16], h, t % 16, as_type(row, kind)[1])
    return c


@pytest.mark.parametrize("at", [[0], [40], [329], [3, 70, 200]])
@pytest.mark.parametrize("kind,big,small,away", [("f16", 1e4, 1e-4, 45.0), ("bf16", 1e20, 1.0, 70.0), ("bf16", 1e30, 1e-3, 80.0)])
@pytest.mark.parametrize("group,dim", [(1, 64), (1, 128), (2, 128), (4, 128), (8, 64)])
def test_large_values_that_are_not_attended(kind, big, small, away, group, dim, at):
    check_decode_and_mass(shunned(kind, group, dim, at, big, small, away), (0, 64))


@pytest.mark.parametrize("group", [2, 4, 8])
def test_heads_that_attend_to_values_of_different_sizes(group):
    check_decode_and_mass(shunned("bf16", group, 128, [10, 100], 1e20, 1.0, 70.0, heads=2, turned=True), (0, 64))


@pytest.mark.parametrize("kind,ratio", [("f16", 2.0 ** 24), ("bf16", 2.0 ** 60), ("bf16", 2.0 ** -60)])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
def test_groups_of_different_sizes(kind, ratio, group):
    """A row's two groups of 64 dimensions, one far larger than the other."""
    size = np.where(np.arange(128) < 64, 2.0 ** -12, 2.0 ** -12 * ratio)[None].repeat(200, 0)
    check_decode_and_mass(decode_case(group, [200], 2, group, 128, kind, sized(np.full(200, 1.0), size)), (0, 64))


# ---- the ends of the type's range -----------------------------------------------------------------

@pytest.mark.parametrize("size", [1e-37, 3e-36, 1e-33, 8e37])
@pytest.mark.parametrize("group", [1, 2, 4])
def test_values_at_the_ends_of_the_range(size, group):
    """bf16 values near the smallest normal numbers, and so near the largest that their sum is not finite."""
    def spread(rng, n, heads, dim):
        return size * np.sign(rng.standard_normal((1, heads, dim))) * (1 + rng.random((n, heads, dim)))

    rows = iter([lambda rng, n, h, d: rng.standard_normal((n, h, d)), spread])
    c = decode_case(group, [300, 40], 2, group, 64, "bf16", lambda *a: next(rows)(*a))
    check_decode_and_mass(c)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("group,dim", [(1, 64), (2, 128), (8, 128)])
def test_one_token_returns_its_value(kind, group, dim):
    """A single weight is 1: the output is the held value, rounded once to the type."""
    c = decode_case(group, [1, 1, 1], 2, group, dim, kind, sized(np.full(3, 30.0), [1.0, 100.0, 1e-3]))
    v = oc.values(c["vp"], dim)[c["tables"][:, 0], :, 0]
    want = torch.from_numpy(v).to(TYPES[kind][0]).repeat_interleave(group, 1)
    assert torch.equal(run_decode(c).cpu(), want)


@pytest.mark.parametrize("k_size", [3e37, 1e34, 1e30, 1e-30, 3e-36])
@pytest.mark.parametrize("heads,group,dim", [(1, 1, 64), (2, 1, 128), (3, 2, 64), (2, 4, 128), (1, 8, 128)])
def test_keys_at_the_ends_of_the_range(k_size, heads, group, dim):
    """Keys near the ends of bf16's range with queries near the other one: ordinary scores."""
    c = decode_case(group * dim, [200, 17], heads, group, dim, "bf16", sized(np.full(217, k_size), np.full(217, 1.0)))
    c["q"], c["qx"] = as_type(c["qx"] / k_size, "bf16")
    check_decode_and_mass(c, (0, 64))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,group", [(1, 1), (6, 1), (3, 2), (1, 4), (4, 4), (2, 8)])
def test_weights_keep_their_precision(heads, group, dim):
    """fp16 values whose sum nearly cancels: what the weights' rounding leaves shows. Small scores keep e below it."""
    lengths = [2, 5, 16, 33, 64, 100]
    check_decode_and_mass(decode_case(heads + dim, lengths, heads, group, dim, "f16", sized(np.full(220, 0.05), np.full(220, 1.0))), (0, 16))


# ---- signs, zeros and NaN in every head layout -----------------------------------------------------

LAYOUTS = [(1, 1, 64), (5, 1, 128), (2, 2, 64), (3, 2, 128), (2, 4, 64), (1, 4, 128), (1, 8, 64), (4, 8, 128)]


@pytest.mark.parametrize("scale", [0.0, -0.125, 3.0])
@pytest.mark.parametrize("heads,group,dim", LAYOUTS)
def test_scales_of_any_sign(scale, heads, group, dim):
    c = decode_case(dim + group, [100, 17, 64, 1], heads, group, dim, "f16", sized(np.full(182, 0.1), np.full(182, 1.0)))
    check_decode_and_mass(dict(c, scale=scale), (0, 32))


@pytest.mark.parametrize("heads,group,dim", LAYOUTS)
@pytest.mark.parametrize("partition", [0, 16, 64])
def test_queries_that_are_zero_or_not_finite_stay_with_their_head(heads, group, dim, partition):
    c = decode_case(3 * dim + group, [150, 33], heads, group, dim, "bf16")
    plain = run_decode(c, partition)
    for value, at in ((0.0, 0), (float("nan"), heads * group - 1), (float("inf"), heads * group // 2), (float("-inf"), 0)):
        q = c["q"].clone()
        q[0, at, 5 if value else slice(None)] = value
        got = run_decode(dict(c, q=q), partition)
        others = [h for h in range(heads * group) if h != at]
        assert torch.equal(got[0, others], plain[0, others]) and torch.equal(got[1], plain[1])
        if value == 0.0:  # the mean of the values
            v = oc.values(c["vp"], dim)[c["tables"][0, np.arange(150) // 16], 0, np.arange(150) % 16]
            # the output's rounding, and 150 2^-23 of the sum (weights are exactly 1)
            assert (np.abs(got[0, at].double().cpu().numpy() - v.mean(0)) <= 2.0 ** -8 * np.abs(v.mean(0)) + 2.0 ** -14 * np.abs(v).mean(0)).all()
        else:
            assert torch.isnan(got[0, at]).all()


@pytest.mark.parametrize("heads,group", [(2, 1), (3, 2), (1, 4), (2, 8)])
@pytest.mark.parametrize("partition", [0, 16])
def test_values_that_are_not_finite_stay_with_their_group(heads, group, partition):
    c = decode_case(90 + group, [70, 20], heads, group, 128, "f16")
    plain = run_decode(c, partition)
    row = oc.values(c["vp"], 128)[c["tables"][0, 2], heads - 1, 7].copy()
    row[70] = np.inf
    oc.store_row(c["vp"], c["tables"][0, 2], heads - 1, 7, row)
    got = run_decode(c, partition)
    hit = slice((heads - 1) * group, None)
    assert torch.isnan(got[0, hit, 64:]).all() and torch.equal(got[0, hit, :64], plain[0, hit, :64])
    assert torch.equal(got[0, :(heads - 1) * group], plain[0, :(heads - 1) * group]) and torch.equal(got[1], plain[1])


@pytest.mark.parametrize("heads,group,dim", LAYOUTS)
def test_scores_beyond_whole_numbers_steps(heads, group, dim):
    """Scores of 2^25 and more, whose neighbours in fp32 lie 4 apart, with values near the type's largest: one token
    takes all the weight, whichever it is, and the output is its value."""
    c = decode_case(group + dim, [90], heads, group, dim, "bf16", sized(np.full(90, 1.0), np.full(90, 2e37)))
    base = np.sign(np.random.default_rng(5).standard_normal(dim))
    c["q"], c["qx"] = as_type(np.tile(base, (1, heads * group, 1)), "bf16")
    order = np.random.default_rng(6).permutation(90)  # rising and falling, far apart: 2^18 and more between any two
    for t in range(90):
        for h in range(heads):
            oc.store_row(c["kp"], c["tables"][0, t // 16], h, t % 16, as_type((2.0 ** 18 + 2.0 ** 13 * order[t]) * base, "bf16")[1])
    c["scale"] = 16.0
    k = oc.values(c["kp"], dim)[c["tables"][0, np.arange(90) // 16], :, np.arange(90) % 16]
    x = np.einsum("thd,d->ht", k, base)
    first = x.argmax(1)
    assert ((x == x.max(1, keepdims=True)).sum(1) == 1).all()
    v = oc.values(c["vp"], dim)[c["tables"][0, first // 16], np.arange(heads), first % 16]
    want = torch.from_numpy(v).to(torch.bfloat16).repeat_interleave(group, 0)
    for partition in (0, 16, 64):
        assert torch.equal(run_decode(c, partition)[0].cpu(), want)
