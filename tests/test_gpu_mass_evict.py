"""Gathered attention weight and eviction by it, on the GPU against the fp64 oracle.

Tolerance of the mass: a weight's score is an fp32 sum of D products, off by at most
e := D 2^-24 scale sum |q k| (for 4-bit pools with |k| as s (n + |z|)); the weight
then is off by a factor of 1 + 2 e + 2^-21 (score and softmax sum, exponential and
logarithm), and the sum over H heads and the decay add at most (H + 2) 2^-24.  A
logarithm of the softmax sum of size up to 2^5 held in fp32 adds 2^-19.
Eviction moves bytes and selects by comparisons: everything is equal, bit for bit.
"""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_478_b200 as pa
from oracle import compress as oc
from paged_kv_cache_478_b200 import synthetic as syn
from tests.test_gpu_q4 import cuda, decode_case, random_rows

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "q4_f16": torch.float16, "q4_bf16": torch.bfloat16}
CODE = {"f32": pa.PA_F32, "f16": pa.PA_F16, "bf16": pa.PA_BF16, "q4_f16": pa.PA_Q4_F16, "q4_bf16": pa.PA_Q4_BF16}


@pytest.fixture(autouse=True)
def _clean_error_word():
    if torch.cuda.is_available():
        pa.pa_device_errors()
    yield


def wide_case(seed, lengths, heads, group, dim, kind):
    """A decode problem over a 16- or 32-bit pool, NaN outside the cached tokens."""
    rng = np.random.default_rng(seed)
    need = [-(-n // 16) for n in lengths]
    nb, wide = sum(need) + 1, max(need + [1])
    tables = syn.random_tables(rng, lengths, nb, wide)
    k = torch.full((nb, heads, 16, dim), float("nan"), dtype=TORCH[kind])
    v = k.clone()
    for s, n in enumerate(lengths):
        for t in range(n):
            b = tables[s, t // 16]
            k[b, :, t % 16] = torch.from_numpy(rng.standard_normal((heads, dim))).to(TORCH[kind])
            v[b, :, t % 16] = torch.from_numpy(rng.standard_normal((heads, dim))).to(TORCH[kind])
    q = torch.from_numpy(rng.standard_normal((len(lengths), heads * group, dim))).to(TORCH[kind])
    return dict(k=k.cuda(), v=v.cuda(), kx=k.double().numpy(), vx=v.double().numpy(), mag=k.double().abs().numpy(), q=q.cuda(), qx=q.double().numpy(),
                tables=tables, lens=np.array(lengths, dtype=np.int32), heads=heads, group=group, dim=dim, kind=kind, scale=1 / math.sqrt(dim))


def any_case(seed, lengths, heads, group, dim, kind):
    if not kind.startswith("q4"):
        return wide_case(seed, lengths, heads, group, dim, kind)
    c = decode_case(seed, lengths, heads, group, dim, kind[3:])
    n, s, z = oc.parts(c["kp"], dim)
    return dict(c, kind=kind, k=cuda(c["kp"]), v=cuda(c["vp"]), kx=oc.values(c["kp"], dim), vx=oc.values(c["vp"], dim),
                mag=np.repeat(s, 64, -1) * (n + np.abs(np.repeat(z, 64, -1))))


def pool_of(c):
    p = pa.pa_pool_create(c["k"].shape[0], 16, c["heads"], c["dim"], CODE[c["kind"]])
    return pa.pa_pool_set_query_heads(p, c["heads"] * c["group"])


def mass_workspace(pool, S, blocks, partition=0, longest=0):
    return torch.empty(pa.pa_decode_mass_workspace_bytes(pool, S, blocks, longest, partition), dtype=torch.uint8, device="cuda")


LENGTHS = [0, 1, 16, 17, 130, 300]


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16", "q4_f16", "q4_bf16"])
@pytest.mark.parametrize("heads,group,dim", [(1, 1, 64), (6, 1, 128), (3, 2, 64), (2, 8, 128)])
def test_mass_against_the_definition(kind, heads, group, dim):
    c = any_case(heads * 10 + group, LENGTHS, heads, group, dim, kind)
    pool, S, HQ = pool_of(c), len(LENGTHS), heads * group
    _, weights, _ = oc.attend(c["qx"], c["kx"], np.nan_to_num(c["vx"]), c["lens"], c["tables"], c["scale"])
    stride = c["tables"].shape[1] * 16 + 5
    before = torch.rand((S, stride), device="cuda")
    bt, cl = cuda(c["tables"]), cuda(c["lens"])
    want = oc.gather_mass(before.double().cpu().numpy(), weights, 0.75)
    e = max(dim * 2.0 ** -24 * c["scale"] * (np.abs(c["qx"][s, h]) @ c["mag"][c["tables"][s, t // 16], h // group, t % 16])
            for s, L in enumerate(LENGTHS) for t in range(L) for h in range(HQ))
    rel = 2 * e + 2.0 ** -21 + (HQ + 2) * 2.0 ** -24 + 2.0 ** -19
    plain = torch.empty_like(c["q"])
    for partition in (0, 64):
        ws = mass_workspace(pool, S, bt.shape[1], partition)
        pa.pa_decode_attention(pool, c["q"], c["k"], c["v"], bt, cl, c["scale"], plain, ws, partition_size=partition)
        out, after = torch.full_like(c["q"], float("nan")), torch.full_like(before, -1.0)
        pa.pa_decode_attention_mass(pool, c["q"], c["k"], c["v"], bt, cl, c["scale"], out, before, after, ws, decay=0.75, partition_size=partition)
        assert pa.pa_device_errors() == 0
        assert torch.equal(out, plain)
        got = after.double().cpu().numpy()
        for s, L in enumerate(LENGTHS):
            assert (np.abs(got[s, :L] - want[s, :L]) <= rel * want[s, :L]).all()
            assert (got[s, L:] == -1).all()
        # in place, planned, on another stream; twice the same bits
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            inplace = before.clone()
            pa.pa_decode_plan(pool, cl, bt.shape[1], ws, partition_size=partition)
            pa.pa_decode_attention_mass_planned(pool, c["q"], c["k"], c["v"], bt, c["scale"], out, inplace, inplace, ws, decay=0.75,
                                                partition_size=partition)
        side.synchronize()
        for s, L in enumerate(LENGTHS):
            assert torch.equal(inplace[s, :L], after[s, :L]) and torch.equal(inplace[s, L:], before[s, L:])
        # no mass_in: the weights alone, which sum to the number of query heads
        alone = torch.zeros_like(before)
        pa.pa_decode_attention_mass(pool, c["q"], c["k"], c["v"], bt, cl, c["scale"], out, None, alone, ws, partition_size=partition)
        sums = alone.double().sum(1).cpu().numpy()
        assert (np.abs(sums - HQ * (c["lens"] > 0)) <= rel * HQ).all()


def test_mass_planned_needs_its_plan():
    c = wide_case(3, [20], 2, 1, 64, "f16")
    pool = pool_of(c)
    ws = mass_workspace(pool, 1, 2)
    mass = torch.zeros((1, 32), device="cuda")
    with pytest.raises(pa.PagedAttnError) as err:
        pa.pa_decode_attention_mass_planned(pool, c["q"], c["k"], c["v"], cuda(c["tables"]), c["scale"], torch.empty_like(c["q"]), None, mass, ws)
    assert err.value.status == 1
    small = torch.empty(pa.pa_decode_workspace_bytes(pool, 1, 2), dtype=torch.uint8, device="cuda")
    with pytest.raises(pa.PagedAttnError) as err:
        pa.pa_decode_attention_mass(pool, c["q"], c["k"], c["v"], cuda(c["tables"]), cuda(c["lens"]), c["scale"], torch.empty_like(c["q"]), None,
                                    mass, small)
    assert err.value.status == 6
    assert not mass.any()


def test_mass_of_a_stale_plan_touches_nothing():
    c = wide_case(4, [20], 2, 1, 64, "f16")
    pool = pool_of(c)
    ws = mass_workspace(pool, 1, 2)
    pa.pa_decode_plan(pool, cuda(c["lens"]), 2, ws)
    torch.cuda.synchronize()
    ws.zero_()
    mass, out = torch.full((1, 32), 2.0, device="cuda"), torch.full_like(c["q"], 7.0)
    pa.pa_decode_attention_mass_planned(pool, c["q"], c["k"], c["v"], cuda(c["tables"]), c["scale"], out, None, mass, ws)
    assert pa.pa_device_errors() == pa.PA_DEVERR_PLAN
    assert (mass == 2).all() and (out == 7).all()


@pytest.mark.parametrize("group", [1, 2, 8])
def test_mass_over_a_long_cache_of_zeros(group):
    """K and V all zero (scale 0): every weight is 1 / L, however long the cache.  The softmax sum's
    logarithm, below 2^7 + 2^7, and its reference are fp32: off by 2^-17 each, a weight by 2^-16."""
    L, dim = 300001, 64
    blocks = -(-L // 16)
    pool = pa.pa_pool_set_query_heads(pa.pa_pool_create(blocks, 16, 1, dim, pa.PA_Q4_BF16), group)
    k = torch.zeros((blocks, 1, 9 * dim), dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    q = torch.ones((1, group, dim), dtype=torch.bfloat16, device="cuda")
    out, mass = torch.full_like(q, 7), torch.full((1, blocks * 16), -1.0, device="cuda")
    tables = torch.arange(blocks, dtype=torch.int32, device="cuda")[None]
    ws = mass_workspace(pool, 1, blocks)
    pa.pa_decode_attention_mass(pool, q, k, v, tables, cuda(np.array([L], dtype=np.int32)), 0.125, out, None, mass, ws)
    assert (out == 0).all() and (mass[0, L:] == -1).all()
    assert ((mass[0, :L] * L / group - 1).abs() <= 2.0 ** -16).all()


# ---- eviction --------------------------------------------------------------------------

def evict_state(rng, lengths, keeps, stride, ties=False):
    S = len(lengths)
    mass = np.exp(2 * rng.standard_normal((S, stride))).astype(np.float32)
    if ties:
        mass = rng.integers(0, 3, (S, stride)).astype(np.float32)
        mass[rng.random(mass.shape) < 0.1] = -0.0
    mass[rng.random(mass.shape) < 0.02] = np.nan
    mass[rng.random(mass.shape) < 0.02] = np.inf
    held = [min(n, int(rng.integers(0, n + 1))) for n in lengths]
    history = np.array([[h, 2 * h + int(rng.integers(0, 5)) if h else 0] for h in held], dtype=np.int32)
    positions = np.sort(rng.integers(0, 2 * stride, (S, stride)), axis=1).astype(np.int32)
    return mass, positions, history


def run_evict(c, keeps, sinks, recent, state, inplace, k=None, v=None):
    pool = pool_of(dict(c, group=1))
    mass, positions, history = (cuda(x) for x in state)
    track = dict(mass=mass, positions=positions, history=history)
    after = track if inplace else {n: torch.full_like(t, -9) for n, t in track.items()}
    ws = torch.empty(pa.pa_evict_workspace_bytes(pool, len(c["lens"]), c["tables"].shape[1]), dtype=torch.uint8, device="cuda")
    pa.pa_evict_tokens(pool, k, v, cuda(c["tables"]), cuda(c["lens"]), cuda(np.array(keeps, dtype=np.int32)), sinks, recent, track, after, ws)
    return after


def rows_of(pool, dim):
    """Every token row of a pool as bytes [NB, H, 16, bytes]."""
    a = pool.cpu()
    if a.dtype == torch.uint8:
        data = a[..., :8 * dim].reshape(*a.shape[:2], dim // 32, 16, 16).permute(0, 1, 3, 2, 4).flatten(3)
        word = a[..., 8 * dim:].reshape(*a.shape[:2], dim // 64, 16, 4).permute(0, 1, 3, 2, 4).flatten(3)
        return torch.cat([data, word], 3).numpy().copy()
    return a.contiguous().view(torch.uint8).reshape(*a.shape[:3], -1).numpy().copy()


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16", "q4_f16", "q4_bf16"])
@pytest.mark.parametrize("heads,dim", [(1, 64), (3, 128)])
@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("sinks,recent,ties", [(0, 0, True), (4, 37, False), (500, 500, False), (1, 1, True)])
def test_evict_is_exact(kind, heads, dim, inplace, sinks, recent, ties):
    rng = np.random.default_rng(heads + sinks + recent)
    lengths = [0, 1, 17, 40, 64, 333, 1030, 2100]
    keeps = [0, 0, 5, 40, 1, 200, 1029, 700]
    c = any_case_bytes(rng, lengths, heads, dim, kind)
    stride = c["tables"].shape[1] * 16 + (0 if inplace else 3)
    state = evict_state(rng, lengths, keeps, stride, ties)
    k, v = c["k"].clone(), c["v"].clone()
    after = run_evict(c, keeps, sinks, recent, state, inplace, k, v)
    assert pa.pa_device_errors() == 0
    want = [rows_of(c["k"], dim), rows_of(c["v"], dim)]
    for s, (L, keep) in enumerate(zip(lengths, keeps)):
        moves, mass, positions, history = oc.evict(state[0][s], state[1][s], state[2][s], L, keep, sinks, recent)
        for a, b in moves:
            for w in want:
                w[c["tables"][s, b // 16], :, b % 16] = w[c["tables"][s, a // 16], :, a % 16]
        got = {n: t[s].cpu().numpy() for n, t in after.items()}
        left = min(L, keep)
        assert np.array_equal(got["mass"][:L], np.array(mass[:L], dtype=np.float32), equal_nan=True)
        assert np.array_equal(got["positions"][:left], positions[:left])
        assert tuple(got["history"]) == history
        tail = state[0][s] if inplace else np.full(stride, -9, dtype=np.float32)
        assert np.array_equal(got["mass"][L:], tail[L:], equal_nan=True)
    assert np.array_equal(rows_of(k, dim), want[0]) and np.array_equal(rows_of(v, dim), want[1])


def any_case_bytes(rng, lengths, heads, dim, kind):
    """Pools of random bytes: eviction moves them as they are."""
    need = [-(-n // 16) for n in lengths]
    nb, wide = sum(need) + 1, max(need + [1])
    tables = syn.random_tables(rng, lengths, nb, wide)
    if kind.startswith("q4"):
        mk = lambda: cuda(rng.integers(0, 256, (nb, heads, 9 * dim)).astype(np.uint8))  # noqa: E731
    else:
        size = 4 if kind == "f32" else 2
        mk = lambda: cuda(rng.integers(0, 256, (nb, heads, 16, dim * size)).astype(np.uint8)).view(TORCH[kind])  # noqa: E731
    return dict(k=mk(), v=mk(), tables=tables, lens=np.array(lengths, dtype=np.int32), heads=heads, dim=dim, kind=kind, group=1)


def test_evict_of_a_long_sequence():
    rng = np.random.default_rng(8)
    for L, keep, recent in [(40000, 9000, 1000), (70000, 69999, 0), (33000, 1, 0)]:
        c = any_case_bytes(rng, [L], 1, 64, "q4_f16")
        stride = c["tables"].shape[1] * 16
        state = evict_state(rng, [L], [keep], stride)
        k, v = c["k"].clone(), c["v"].clone()
        after = run_evict(c, [keep], 4, recent, state, False, k, v)
        moves, mass, positions, history = oc.evict(state[0][0], state[1][0], state[2][0], L, keep, 4, recent)
        assert np.array_equal(after["mass"][0, :L].cpu().numpy(), np.array(mass[:L], dtype=np.float32), equal_nan=True)
        assert np.array_equal(after["positions"][0, :keep].cpu().numpy(), positions[:keep])
        want = rows_of(c["k"], 64)
        src, dst = np.array([m[0] for m in moves]), np.array([m[1] for m in moves])
        if len(moves):
            want[c["tables"][0, dst // 16], :, dst % 16] = want[c["tables"][0, src // 16], :, src % 16]
        assert np.array_equal(rows_of(k, 64), want)


@pytest.mark.parametrize("inplace", [False, True])
def test_evict_of_everything(inplace):
    """keep 0: no pass of the selection runs, and nothing moves."""
    rng = np.random.default_rng(81)
    lengths = [5000, 1, 0, 33, 17000] * 20  # clusters of 8 CTAs each
    c = any_case_bytes(rng, lengths, 1, 64, "f16")
    stride = c["tables"].shape[1] * 16
    state = evict_state(rng, lengths, [0] * len(lengths), stride)
    for sinks, recent in ((0, 0), (4, 64)):
        k, v = c["k"].clone(), c["v"].clone()
        after = run_evict(c, [0] * len(lengths), sinks, recent, state, inplace, k, v)
        assert pa.pa_device_errors() == 0
        got = after["mass"].cpu().numpy()
        for s, L in enumerate(lengths):
            h, nxt = state[2][s]
            assert (got[s, :L] == 0).all()
            assert after["history"][s].tolist() == ([0, nxt + L - h] if L else [h, nxt])
        assert torch.equal(k.view(torch.int16), c["k"].view(torch.int16))
        assert torch.equal(v.view(torch.int16), c["v"].view(torch.int16))


def test_evict_reports_bad_lengths_and_blocks():
    rng = np.random.default_rng(9)
    c = any_case_bytes(rng, [40, 40, 40], 2, 64, "f16")
    state = evict_state(rng, [40] * 3, [10] * 3, 48)
    k, v = c["k"].clone(), c["v"].clone()
    c["lens"][0] = 1000  # past the table: clamped to its 48 slots
    run_evict(c, [48, -1, 40], 0, 0, state, False, k, v)
    assert pa.pa_device_errors() == pa.PA_DEVERR_CONTEXT_LEN
    assert np.array_equal(rows_of(k, 64), rows_of(c["k"], 64))
    c["lens"][0] = 40
    c["tables"][1] = 10 ** 6
    run_evict(c, [40, 10, 40], 0, 0, state, False, k, v)
    assert pa.pa_device_errors() == pa.PA_DEVERR_BLOCK_ID
    assert np.array_equal(rows_of(k, 64), rows_of(c["k"], 64))


def test_a_repeated_call_repeats_its_moves_and_replays_in_a_graph():
    rng = np.random.default_rng(10)
    c = any_case_bytes(rng, [100, 64], 2, 128, "bf16")
    pool = pool_of(c)
    state = evict_state(rng, [100, 64], [30, 30], 112)
    track = dict(zip(("mass", "positions", "history"), (cuda(x) for x in state)))
    after = {n: torch.zeros_like(t) for n, t in track.items()}
    ws = torch.empty(pa.pa_evict_workspace_bytes(pool, 2, 7), dtype=torch.uint8, device="cuda")
    bt, cl, keep = cuda(c["tables"]), cuda(c["lens"]), cuda(np.array([30, 30], dtype=np.int32))
    k, v = c["k"].clone(), c["v"].clone()
    call = lambda: pa.pa_evict_tokens(pool, k, v, bt, cl, keep, 1, 3, track, after, ws)  # noqa: E731
    call()
    once = (k.clone(), v.clone(), {n: t.clone() for n, t in after.items()})
    call()
    same = lambda: all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in  # noqa: E731
                       [(k, once[0]), (v, once[1])] + [(after[n], once[2][n]) for n in after])
    assert same()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call()
    for _ in range(2):
        k.copy_(c["k"])
        v.copy_(c["v"])
        g.replay()
        torch.cuda.synchronize()
        assert same()


# ---- the operators together, as a server would use them -----------------------------------

@pytest.mark.parametrize("kind", ["f16", "q4_bf16"])
def test_decode_gather_evict_loop(kind):
    """Steps of append, attend + gather, and eviction when over budget, with the block manager;
    at every step the attention equals the oracle's over the tokens that are still cached, and
    the track says which those are."""
    rng = np.random.default_rng(12)
    S, heads, group, dim, budget, slack = 3, 2, 2, 64, 40, 12
    HQ, nb, wide = heads * group, 40, 6
    dt = TORCH[kind]
    bm = pa.BlockManager(nb)
    pool = pa.pa_pool_set_query_heads(pa.pa_pool_create(nb, 16, heads, dim, CODE[kind]), HQ)
    shape = (nb, heads, 9 * dim) if kind.startswith("q4") else (nb, heads, 16, dim)
    k = torch.full(shape, 255, dtype=torch.uint8, device="cuda") if kind.startswith("q4") else torch.full(shape, float("nan"), dtype=dt, device="cuda")
    v = k.clone()
    tables, lens = np.full((S, wide), -1, dtype=np.int32), np.zeros(S, dtype=np.int32)
    track = dict(mass=torch.zeros((S, wide * 16), device="cuda"), positions=torch.zeros((S, wide * 16), dtype=torch.int32, device="cuda"),
                 history=torch.zeros((S, 2), dtype=torch.int32, device="cuda"))
    ws = mass_workspace(pool, S, wide)
    ews = torch.empty(pa.pa_evict_workspace_bytes(pool, S, wide), dtype=torch.uint8, device="cuda")
    keep = torch.full((S,), budget, dtype=torch.int32, device="cuda")
    seen_k = [np.zeros((0, heads, dim)) for _ in range(S)]  # every token ever, by position
    seen_v = [np.zeros((0, heads, dim)) for _ in range(S)]

    def stored(x):  # what the pool holds of a row
        if not kind.startswith("q4"):
            return x
        n, s, z = oc.quantise(x)
        return np.repeat(s, 64, -1) * (n - np.repeat(z, 64, -1))

    evictions = 0
    for step in range(40):
        new = [int(rng.integers(1, 4)) if step else 30 for _ in range(S)]
        slots, kn, vn = [], [], []
        for s in range(S):
            lens[s], sl, pairs = bm.append_tokens(tables[s], int(lens[s]), new[s])
            assert len(pairs) == 0
            a, b = torch.from_numpy(rng.standard_normal((2, new[s], heads, dim))).to(dt)
            slots.append(sl), kn.append(a), vn.append(b)
            seen_k[s] = np.concatenate([seen_k[s], stored(a.double().numpy())])
            seen_v[s] = np.concatenate([seen_v[s], stored(b.double().numpy())])
        pa.pa_reshape_and_cache(pool, torch.cat(kn).cuda(), torch.cat(vn).cuda(), cuda(np.concatenate(slots)), k, v)
        q = torch.from_numpy(rng.standard_normal((S, HQ, dim))).to(dt).cuda()
        out = torch.empty_like(q)
        bt, cl = cuda(tables), cuda(lens)
        pa.pa_decode_attention_mass(pool, q, k, v, bt, cl, 0.2, out, track["mass"], track["mass"], ws, decay=0.9)
        assert pa.pa_device_errors() == 0
        hist, pos = track["history"].cpu().numpy(), track["positions"].cpu().numpy()
        for s in range(S):
            L, (held, nxt) = int(lens[s]), hist[s]
            at = [int(pos[s, t]) if t < held else int(nxt + t - held) for t in range(L)]
            assert len(set(at)) == L
            for h in range(HQ):
                kx, vx = seen_k[s][at, h // group], seen_v[s][at, h // group]
                x = 0.2 * kx @ q[s, h].double().cpu().numpy()
                w = np.exp(x - x.max())
                w /= w.sum()
                assert np.abs(out[s, h].double().cpu().numpy() - w @ vx).max() <= 2.0 ** -7 * np.abs(vx).max()
        if lens.max() > budget + slack:
            evictions += 1
            pa.pa_evict_tokens(pool, k, v, bt, cl, keep, 2, 8, track, track, ews)
            for s in range(S):
                used, left = -(-int(lens[s]) // 16), -(-min(int(lens[s]), budget) // 16)
                if used > left:
                    bm.release_table(tables[s, left:used].copy(), used - left)
                    tables[s, left:used] = -1
                lens[s] = min(int(lens[s]), budget)
            pos = track["positions"].cpu().numpy()
            total = [len(x) for x in seen_k]
            for s in range(S):
                if track["history"][s, 0] == lens[s] == budget:
                    kept = set(pos[s, :budget].tolist())
                    assert {0, 1} <= kept and set(range(total[s] - 8, total[s])) <= kept
    assert evictions >= 3


@pytest.mark.parametrize("kind", ["f32", "bf16", "q4_f16"])
def test_mass_in_a_graph(kind):
    """Plan, attention and gathering captured together and replayed: every replay decays and adds once more."""
    c = any_case(21, [40, 0, 333], 2, 2 if kind != "f32" else 1, 64, kind)
    pool = pool_of(c)
    bt, cl = cuda(c["tables"]), cuda(c["lens"])
    ws = mass_workspace(pool, 3, bt.shape[1])
    out, mass = torch.empty_like(c["q"]), torch.zeros((3, bt.shape[1] * 16), device="cuda")
    step = lambda m: pa.pa_decode_attention_mass(pool, c["q"], c["k"], c["v"], bt, cl, c["scale"], out, m, m, ws, decay=0.5)  # noqa: E731
    want = torch.zeros_like(mass)
    for _ in range(3):
        step(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step(mass)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(mass, want) and pa.pa_device_errors() == 0


def test_evict_of_a_very_long_sequence():
    """More keys than the cluster's shared memory holds: the track is read anew each pass."""
    rng = np.random.default_rng(22)
    L, keep = 400001, 123457
    c = any_case_bytes(rng, [L], 1, 64, "q4_bf16")
    state = evict_state(rng, [L], [keep], c["tables"].shape[1] * 16, ties=True)
    for inplace in (False, True):
        k, v = c["k"].clone(), c["v"].clone()
        after = run_evict(c, [keep], 4, 5000, state, inplace, k, v)
        moves, mass, positions, history = oc.evict(state[0][0], state[1][0], state[2][0], L, keep, 4, 5000)
        assert np.array_equal(after["mass"][0, :L].cpu().numpy(), np.array(mass[:L], dtype=np.float32), equal_nan=True)
        assert np.array_equal(after["positions"][0, :keep].cpu().numpy(), positions[:keep])
        assert tuple(after["history"][0].cpu().numpy()) == history
        want = rows_of(c["k"], 64)
        src, dst = np.array([m[0] for m in moves]), np.array([m[1] for m in moves])
        want[c["tables"][0, dst // 16], :, dst % 16] = want[c["tables"][0, src // 16], :, src % 16]
        assert np.array_equal(rows_of(k, 64), want)


def test_evict_offsets_past_32_bits():
    """Rows moved in the last blocks of a pool of more than 2^32 bytes."""
    rng = np.random.default_rng(23)
    heads, dim, nb = 32, 128, 34000
    c = any_case_bytes(rng, [90], heads, dim, "f16")
    small = c["k"].shape[0]
    state = evict_state(rng, [90], [30], 96)
    k, v = c["k"].clone(), c["v"].clone()
    run_evict(c, [30], 1, 5, state, False, k, v)
    big_k = torch.zeros((nb, heads, 16, dim), dtype=torch.float16, device="cuda")
    assert big_k.numel() * 2 > 2 ** 32
    big_v = torch.zeros_like(big_k)
    big_k[-small:], big_v[-small:] = c["k"], c["v"]
    far = dict(c, k=big_k, tables=np.where(c["tables"] >= 0, c["tables"] + nb - small, -1).astype(np.int32))
    run_evict(far, [30], 1, 5, state, False, big_k, big_v)
    assert torch.equal(big_k[-small:].view(torch.uint8), k.view(torch.uint8))
    assert torch.equal(big_v[-small:].view(torch.uint8), v.view(torch.uint8)) and not big_k[:-small].any()
