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
