"""pa_decode_mod on the CPU: its refusals, and its restatement against plain
decode, against scalar loops and against invariants."""

import math

import numpy as np
import pytest
import torch

import oracle
from oracle import modified
from paged_kv_cache_292_gb300 import binding
from paged_kv_cache_292_gb300 import build as pa_build

INVALID, UNSUPPORTED = binding.PA_ERR_INVALID_ARG, binding.PA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return binding.load()


def _args(fp8, **kw):
    a = dict(out=16, query=16, k_cache=16, v_cache=16, block_tables=16, context_lens=16, num_seqs=1, num_queries=1,
             num_heads=8, num_kv_heads=8, head_size=128, block_size=16, max_blocks_per_seq=4, scale=0.1, k_scale=1.0,
             v_scale=1.0, softcap=0.0, alibi_slopes=None, window=0, first_tokens=None, prefix_lens=None, stream=0,
             dtype=binding.PA_BF16, num_physical_blocks=0, workspace=None, workspace_bytes=0, num_ranges=0,
             error_flag=None)
    a.update(kw)
    for name in ("dtype",) if fp8 else ("k_scale", "v_scale"):
        del a[name]
    return list(a.values())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw, code", [
    *[({name: None}, INVALID) for name in ("out", "query", "k_cache", "v_cache", "block_tables", "context_lens")],
    (dict(softcap=-1.0), INVALID),
    (dict(softcap=float("nan")), INVALID),
    (dict(softcap=float("inf")), INVALID),
    (dict(window=-1), INVALID),
    (dict(alibi_slopes=18), INVALID),
    (dict(first_tokens=18), INVALID),
    (dict(prefix_lens=17), INVALID),
    (dict(num_queries=0), INVALID),
    (dict(num_queries=33), UNSUPPORTED),
    (dict(num_heads=72, num_kv_heads=8, num_queries=1), UNSUPPORTED),  # group 9
    (dict(num_heads=32, num_kv_heads=8, num_queries=9), UNSUPPORTED),  # 36 columns
    (dict(num_heads=12), INVALID),
    (dict(head_size=96), UNSUPPORTED),
    (dict(block_size=4097), UNSUPPORTED),
    (dict(scale=float("inf")), INVALID),
    (dict(query=24), INVALID),
    (dict(num_ranges=-1), INVALID),
])
def test_rejects_bad_arguments_on_host(lib, fp8, kw, code):
    fn = lib.pa_decode_fp8_mod if fp8 else lib.pa_decode_mod
    assert fn(*_args(fp8, **kw)) == code
    assert lib.pa_last_error().decode()


def test_types(lib):
    assert lib.pa_decode_mod(*_args(False, dtype=binding.PA_F32, num_queries=2)) == UNSUPPORTED
    assert lib.pa_decode_mod(*_args(False, dtype=binding.PA_FP8_E4M3)) == UNSUPPORTED
    for name in ("k_scale", "v_scale"):
        for bad in (0.0, -1.0, float("nan")):
            assert lib.pa_decode_fp8_mod(*_args(True, **{name: bad})) == INVALID


def test_python_layer_wants_cuda_tensors():
    q = torch.zeros(1, 8, 64)
    pool = torch.zeros(2, 16, 8, 64)
    one = torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.decode_mod(q, pool, pool, one.view(1, 1), one, 0.125, softcap=10.0)


def _batch(seed, S=3, Q=2, H=4, Hk=2, D=4, bs=4, hi=19):
    rng = np.random.default_rng(seed)
    lens = rng.integers(1, hi + 1, S)
    mb = -(-hi // bs)
    tables = rng.permutation(S * mb).reshape(S, mb)
    k, v = rng.standard_normal((2, S * mb, bs, Hk, D))
    return rng.standard_normal((S, Q, H, D)), k, v, tables, lens, bs


@pytest.mark.parametrize("seed", range(3))
def test_restatement_without_modifications_is_plain_decode(seed):
    q, k, v, tables, lens, bs = _batch(seed)
    got, _ = modified.decode_mod(q, k, v, tables, lens, 0.5, bs)
    assert np.allclose(got, oracle.decode_multi(q, k, v, tables, lens, 0.5, bs), atol=1e-12)
    # A window as long as the context and a cap far above the scores change nothing.
    far, _ = modified.decode_mod(q, k, v, tables, lens, 0.5, bs, window=19, softcap=1e7)
    assert np.allclose(got, far, atol=1e-6)


@pytest.mark.parametrize("seed", range(3))
def test_restatement_against_scalar_loops(seed):
    q, k, v, tables, lens, bs = _batch(seed + 10)
    S, Q, H, D = q.shape
    rng = np.random.default_rng(seed)
    slopes, window, cap = rng.standard_normal(H), 5, 1.5
    first, prefix = rng.integers(-2, 9, S), rng.integers(-2, 9, S)
    got, _ = modified.decode_mod(q, k, v, tables, lens, 0.5, bs, softcap=cap, slopes=slopes, window=window,
                                 first=first, prefix=prefix)
    for s in range(S):
        for i in range(Q):
            pos = int(lens[s]) - Q + i
            for h in range(H):
                num, den = [0.0] * D, 0.0
                for t in range(int(lens[s])):
                    sees = pos >= 0 and t >= first[s] and (t < prefix[s] or (t <= pos and pos - t < window))
                    if not sees:
                        continue
                    b, o = int(tables[s, t // bs]), t % bs
                    dot = sum(q[s, i, h, d] * k[b, o, h // 2, d] for d in range(D))
                    w = math.exp(cap * math.tanh(0.5 * dot / cap) - slopes[h] * abs(pos - t))
                    den += w
                    for d in range(D):
                        num[d] += w * v[b, o, h // 2, d]
                want = [x / den for x in num] if den else num
                assert np.allclose(got[s, i, h], want, atol=1e-12)


def test_restatement_ignores_what_nobody_sees():
    q, k, v, tables, lens, bs = _batch(4, Q=1)
    lens[:] = 19
    want, _ = modified.decode_mod(q, k, v, tables, lens, 0.5, bs, window=3)
    k2, v2, t2 = k.copy(), v.copy(), tables.copy()
    for s in range(3):
        for t in range(16):
            k2[tables[s, t // bs], t % bs] = np.nan
            v2[tables[s, t // bs], t % bs] = np.nan
        t2[s, :4] = -1
    got, _ = modified.decode_mod(q, k2, v2, t2, lens, 0.5, bs, window=3)
    assert np.array_equal(got, want)


def test_workspace_size(lib):
    size = binding.pa_decode_mod_workspace_size
    for bad in ((0, 1, 8, 8, 128, 1), (1, 0, 8, 8, 128, 1), (1, 1, 9, 8, 128, 1), (1, 1, 8, 0, 128, 1),
                (1, 1, 8, 8, 0, 1), (1, 1, 8, 8, 128, 3), (1, 1, 8, 8, 128, 1, -1)):
        assert size(*bad) == 0
    # num_ranges partials of (m, l) and O for two slots, and 16 bytes per sequence.
    assert size(5, 3, 8, 2, 64, binding.PA_BF16, 7) >= 7 * 2 * 24 * (8 + 4 * 64) + 16 * 5
