"""Eviction with damaged inputs, on the GPU: the track must go on describing what the
sequence's slots hold.  Everything is equal, bit for bit."""
import numpy as np
import pytest
import torch

import paged_kv_cache_478_b200 as pa
from oracle import compress as oc
from tests.test_gpu_mass_evict import any_case_bytes, evict_state, rows_of, run_evict

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_error_word():
    if torch.cuda.is_available():
        pa.pa_device_errors()
    yield


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("kind", ["f16", "q4_bf16"])
@pytest.mark.parametrize("bad", [[(0, 5)], [(0, 0)], [(1, 2), (1, 9)], [(0, b) for b in range(7)]])
def test_moves_of_bad_blocks_are_dropped_with_their_track(inplace, kind, bad):
    rng = np.random.default_rng(31)
    lengths, keeps = [100, 333, 40], [30, 120, 20]
    c = any_case_bytes(rng, lengths, 3, 64, kind)
    state = evict_state(rng, lengths, keeps, c["tables"].shape[1] * 16)
    damaged = c["tables"].copy()
    for s, b in bad:
        damaged[s, b] = -1 if b % 2 else 10 ** 6
    k, v = c["k"].clone(), c["v"].clone()
    after = run_evict(dict(c, tables=damaged), keeps, 2, 6, state, inplace, k, v)
    want_k, want_v = rows_of(c["k"], 64), rows_of(c["v"], 64)
    dropped = 0
    for s, (L, keep) in enumerate(zip(lengths, keeps)):
        moves, mass, positions, history = oc.evict(state[0][s], state[1][s], state[2][s], L, keep, 2, 6)
        held, nxt = state[2][s]
        for a, b in moves:
            if damaged[s, a // 16] == c["tables"][s, a // 16] and damaged[s, b // 16] == c["tables"][s, b // 16]:
                for w in (want_k, want_v):
                    w[c["tables"][s, b // 16], :, b % 16] = w[c["tables"][s, a // 16], :, a % 16]
            else:  # the destination keeps its own token
                dropped += 1
                mass[b], positions[b] = state[0][s][b], state[1][s][b] if b < held else nxt + b - held
        got = {n: t[s].cpu().numpy() for n, t in after.items()}
        assert np.array_equal(got["mass"][:L], np.array(mass[:L], dtype=np.float32), equal_nan=True)
        assert np.array_equal(got["positions"][:keep], positions[:keep])
        assert tuple(got["history"]) == history
    assert dropped and pa.pa_device_errors() == pa.PA_DEVERR_BLOCK_ID
    assert np.array_equal(rows_of(k, 64), want_k) and np.array_equal(rows_of(v, 64), want_v)


TOP = 2 ** 31 - 1


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("longest", [200, 5000])  # one CTA a sequence, and a cluster of two
def test_a_history_that_does_not_fit_keeps_its_sequence_whole(inplace, longest):
    rng = np.random.default_rng(32)
    bad = [(longest + 1, 2 * longest), (-1, 5), (10, -3), (0, TOP), (TOP, TOP), (-2 ** 31, -2 ** 31), (5, TOP - longest + 6)]
    good = [(longest, 3 * longest), (0, 0), (5, TOP - longest + 5)]
    lengths, keeps = [longest] * (len(bad) + len(good)), [60] * (len(bad) + len(good))
    lengths += [0, 40, 60]  # not over their budget: a stale history does not matter, and nothing is reported for it
    keeps += [0, 40, 61]
    c = any_case_bytes(rng, lengths, 1, 64, "f16")
    mass, positions, history = evict_state(rng, lengths, keeps, c["tables"].shape[1] * 16)
    history[:len(bad) + len(good)] = bad + good
    history[len(bad) + len(good):] = [77, 99]
    state = (mass, positions, history)
    for only_good in (True, False):
        k, v = c["k"].clone(), c["v"].clone()
        lens = np.array(lengths, dtype=np.int32)
        if only_good:
            lens[:len(bad)] = 0
        after = run_evict(dict(c, lens=lens), keeps, 4, 20, state, inplace, k, v)
        assert pa.pa_device_errors() == (0 if only_good else pa.PA_DEVERR_CONTEXT_LEN)
        want = [rows_of(c["k"], 64), rows_of(c["v"], 64)]
        for s, L in enumerate(lens):
            left = keeps[s] if s >= len(bad) else int(L)
            moves, m, p, h = oc.evict(mass[s], positions[s], history[s], int(L), left, 4, 20)
            for a, b in moves:
                for w in want:
                    w[c["tables"][s, b // 16], :, b % 16] = w[c["tables"][s, a // 16], :, a % 16]
            got = {n: t[s].cpu().numpy() for n, t in after.items()}
            assert np.array_equal(got["mass"][:L], np.array(m[:L], dtype=np.float32), equal_nan=True)
            assert np.array_equal(got["positions"][:min(left, L)], p[:min(left, L)]) and tuple(got["history"]) == tuple(h)
        assert np.array_equal(rows_of(k, 64), want[0]) and np.array_equal(rows_of(v, 64), want[1])
