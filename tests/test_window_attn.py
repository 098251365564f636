"""Attention with a sliding window and sinks (infllmv2_window_attn) against the
fp64 oracle, every element.

Bounds, from the roundings of the kernel (half a bf16 step is 2^-8 relative,
half an fp32 step 2^-24):
- a score is an fp32 sum of 128 exact products, then one scaling and the
  exponential's argument: off by at most 136 * 2^-24 * reach =: ds;
- P = exp(s - m) (ex2.approx: 2^-22 relative) is rounded to bf16, so O moves by
  at most (2^-8 + 2 ds + 2^-20) * spread; O itself is rounded once: 2^-8 |O|;
- lse: ds, the logarithm's 2^-21 absolute, the fp32 sum of up to T positive terms
  kept in few partial sums (2^-24 * T / 4 relative), and one rounding of lse.
"""
import numpy as np
import pytest

from oracle import window_oracle as wo
from trainable_block_sparse_compressed_b200 import infllmv2 as host_api

from _helpers import f64

BF, F32 = 2.0 ** -8, 2.0 ** -24


def bounds(O, lse, spread, reach, n_keys):
    ds = 136 * F32 * reach
    eO = (BF + 2 * ds[..., None] + 2.0 ** -20) * spread + BF * np.abs(O) + 1e-30
    eL = ds + 2.0 ** -21 + F32 * n_keys / 4 + 2 * F32 * np.abs(np.where(np.isfinite(lse), lse, 0.0))
    return eO, eL


def check(O, lse, ref, n_keys):
    rO, rL, spread, reach = ref
    eO, eL = bounds(rO, rL, spread, reach, n_keys)
    assert np.isfinite(O).all()
    worst = (np.abs(O - rO) / eO).max(initial=0.0)
    assert worst <= 1.0, f"O is {worst:.3g} times its bound off"
    seen = np.isfinite(rL)
    assert np.array_equal(seen, np.isfinite(lse)) and np.isneginf(lse[~seen]).all()
    worst = (np.abs(lse - rL)[seen] / eL[seen]).max(initial=0.0)
    assert worst <= 1.0, f"lse is {worst:.3g} times its bound off"


def make(B, T, Hq, Hkv, seed, n=3):
    import torch
    g = torch.Generator().manual_seed(seed)
    shapes = [(B, T, Hq, 128), (B, T, Hkv, 128), (B, T, Hkv, 128), (B, T, Hq, 128)]
    return [torch.randn(s, generator=g).to(torch.bfloat16).cuda() for s in shapes[:n]]


def run(api, Q, K, V, window, n_sink, scale=0.0):
    import torch
    B, T, Hq, _ = Q.shape
    p = api.make_params(B, T, Hq, K.shape[2], scale=scale)
    O = torch.full_like(Q, float("nan"))
    lse = torch.full((B, Hq, T), float("nan"), device="cuda")
    api.window_attn(p, window, n_sink, Q, K, V, O, lse)
    assert api.get_status() == 0
    return O, lse


CASES = [
    # B, T, Hq, Hkv, window, n_sink
    (1, 1, 4, 2, 0, 0),          # one token
    (1, 2, 16, 1, 1, 1),
    (2, 127, 2, 2, 0, 0),        # heads of their own
    (1, 128, 4, 2, 64, 4),
    (1, 129, 8, 1, 1, 0),        # each token sees itself alone
    (2, 300, 32, 2, 100, 3),
    (1, 517, 8, 4, 128, 64),
    (1, 640, 8, 8, 333, 0),
    (1, 777, 16, 2, 200, 130),   # sinks past one key tile
    (1, 900, 4, 1, 130, 900),    # every key a sink
    (1, 1000, 32, 2, 5000, 7),   # a window past the sequence
    (1, 1025, 16, 16, 127, 1),
    (3, 1100, 16, 4, 0, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,Hq,Hkv,window,n_sink", CASES)
def test_window_attn_all_elements(cuda_lib, B, T, Hq, Hkv, window, n_sink):
    Q, K, V = make(B, T, Hq, Hkv, seed=T + window)
    O, lse = run(cuda_lib, Q, K, V, window, n_sink)
    q, k, v, o, ls = f64(Q), f64(K), f64(V), f64(O), f64(lse)
    for b in range(B):
        ref = wo.attention(q[b], k[b], v[b], np.arange(T), window, n_sink)
        check(o[b], ls[b].T, ref, T)


@pytest.mark.gpu
def test_window_attn_many_items_per_cta(cuda_lib):
    """More query tile pairs than SMs: rows of the first, middle and last tokens."""
    B, T, Hq, Hkv, window, n_sink = 2, 6001, 32, 2, 700, 64
    Q, K, V = make(B, T, Hq, Hkv, seed=5)
    O, lse = run(cuda_lib, Q, K, V, window, n_sink)
    pos = np.array([0, 1, 63, 64, 699, 700, 701, 763, 764, 765, 2999, 4095, 4096, 5999, 6000])
    for b in range(B):
        ref = wo.attention(f64(Q[b, pos]), f64(K[b]), f64(V[b]), pos, window, n_sink)
        check(f64(O[b, pos]), f64(lse[b][:, pos]).T, ref, window + n_sink)


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,Hq,Hkv,window,n_sink", [
    (2, 1201, 32, 2, 128, 0), (2, 1201, 32, 2, 1, 0), (2, 1333, 32, 2, 256, 64),
    (2, 1333, 32, 2, 257, 3), (2, 2000, 16, 16, 64, 4), (4, 1501, 8, 2, 200, 130),
    (3, 1499, 16, 8, 37, 200),
])
def test_window_attn_short_windows_in_pairs(cuda_lib, B, T, Hq, Hkv, window, n_sink):
    """Windows on both sides of the narrow variant's limit, more query tile
    pairs than SMs: halves of key tiles left out, whole lines written."""
    Q, K, V = make(B, T, Hq, Hkv, seed=T + window)
    O, lse = run(cuda_lib, Q, K, V, window, n_sink)
    pos = np.unique(np.concatenate([np.arange(270), np.arange(270, T, 11), np.arange(T - 40, T)]))
    for b in range(B):
        ref = wo.attention(f64(Q[b, pos]), f64(K[b]), f64(V[b]), pos, window, n_sink)
        check(f64(O[b, pos]), f64(lse[b][:, pos]).T, ref, window + n_sink)


@pytest.mark.gpu
def test_no_window_is_dense_attention(cuda_lib):
    """Within the two kernels' bf16 roundings of P and O."""
    import torch
    api = cuda_lib
    Q, K, V = make(2, 1500, 16, 2, seed=6)
    O, lse = run(api, Q, K, V, 0, 0)
    p = api.make_params(2, 1500, 16, 2)
    Od, ld = torch.empty_like(Q), torch.empty_like(lse)
    api.dense_attn(p, Q, K, V, Od, ld)
    torch.cuda.synchronize()
    assert (lse - ld).abs().max() < 1e-4
    assert (O.float() - Od.float()).abs().max() < 2e-2


@pytest.mark.gpu
def test_window_attn_large_scores_and_scale(cuda_lib):
    """Scores of several hundred (the running maximum moves and O is rescaled)."""
    T, Hq, Hkv, window, n_sink, scale = 700, 8, 2, 300, 5, 0.9
    Q, K, V = make(1, T, Hq, Hkv, seed=7)
    Q = (Q.float() * 3).to(Q.dtype)
    O, lse = run(cuda_lib, Q, K, V, window, n_sink, scale)
    ref = wo.attention(f64(Q)[0], f64(K)[0], f64(V)[0], np.arange(T), window, n_sink, scale)
    check(f64(O)[0], f64(lse)[0].T, ref, T)


@pytest.mark.gpu
def test_window_attn_ignores_keys_outside(cuda_lib):
    """Infinite keys and huge values outside the window and the sinks change
    nothing; a later batch row's do not either."""
    import torch
    T, window, n_sink = 1024, 128, 16
    Q, K, V = make(2, T, 8, 2, seed=8)
    O, lse = run(cuda_lib, Q, K, V, window, n_sink)
    K2, V2 = K.clone(), V.clone()
    K2[0, 128:512] = float("inf")     # outside what tokens >= 640 see, tile aligned
    V2[0, 128:512] = 3e38
    O2, lse2 = run(cuda_lib, Q, K2, V2, window, n_sink)
    assert torch.equal(O[0, 640:], O2[0, 640:]) and torch.equal(lse[0, :, 640:], lse2[0, :, 640:])
    assert torch.equal(O[0, :128], O2[0, :128]) and torch.equal(O[1], O2[1])


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hkv,window,at", [(600, 2, 2, 0, 200), (600, 2, 2, 2, 5), (4100, 32, 2, 100, 3000),
                                                (1000, 16, 4, 64, 999)])
def test_a_value_that_is_not_finite_stays_in_its_sequence_and_head(cuda_lib, T, Hq, Hkv, window, at):
    """Rows that see it are NaN; which rows near it are is not promised, but
    other sequences, other kv heads and all lse are untouched.  An unseen key
    reaches no row at all."""
    import torch
    Q, K, V = make(3, T, Hq, Hkv, seed=T)
    O, lse = run(cuda_lib, Q, K, V, window, 0)
    V2 = V.clone()
    V2[1, at, 0] = float("nan")
    O2, lse2 = run(cuda_lib, Q, K, V2, window, 0)
    G, last = Hq // Hkv, T if window == 0 else min(T, at + window)
    assert torch.isnan(O2[1, at:last, :G]).all()
    assert torch.equal(O2[0], O[0]) and torch.equal(O2[2], O[2]) and torch.equal(lse2, lse)
    assert torch.equal(O2[1, :, G:], O[1, :, G:])
    K2 = K.clone()
    K2[1, T - 1, 0] = float("nan")      # seen by the last token alone
    O3, lse3 = run(cuda_lib, Q, K2, V, window, 0)
    assert torch.equal(O3[:, :T - 1], O[:, :T - 1]) and torch.equal(lse3[..., :T - 1], lse[..., :T - 1])
    assert torch.isnan(O3[1, T - 1, :G]).all() and torch.isnan(lse3[1, :G, T - 1]).all()


@pytest.mark.gpu
def test_window_attn_side_stream_graph_and_repeat(cuda_lib):
    """On a side stream, captured and replayed on new inputs: the same bits."""
    import torch
    api = cuda_lib
    B, T, Hq, Hkv, window, n_sink = 1, 600, 32, 2, 256, 4
    Q, K, V = make(B, T, Hq, Hkv, seed=9)
    O, lse = run(api, Q, K, V, window, n_sink)
    p = api.make_params(B, T, Hq, Hkv)
    Q2, K2, V2 = (torch.zeros_like(x) for x in (Q, K, V))
    O2, lse2 = torch.empty_like(Q), torch.empty_like(lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        api.window_attn(p, window, n_sink, Q2, K2, V2, O2, lse2)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            api.window_attn(p, window, n_sink, Q2, K2, V2, O2, lse2)
    torch.cuda.synchronize()
    Q2.copy_(Q), K2.copy_(K), V2.copy_(V)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    assert api.get_status() == 0


# ---------------------------------------------------------------------------
# refusals (no GPU needed: the host refuses before any launch)
# ---------------------------------------------------------------------------
FAKE = 0x10000


def test_window_attn_refusals():
    import ctypes
    lib = host_api.load()
    call = lambda p, w, s, q=FAKE, o=FAKE: lib.infllmv2_window_attn(  # noqa: E731
        ctypes.byref(p), w, s, q, FAKE, FAKE, o, FAKE, None)
    ok = host_api.make_params(1, 64, 32, 2)
    assert call(ok, -1, 0) == host_api.ERR_INVALID_ARG
    assert call(ok, 0, -1) == host_api.ERR_INVALID_ARG
    assert call(ok, 4, 0, q=None) == host_api.ERR_INVALID_ARG
    assert call(ok, 4, 0, q=FAKE + 8) == host_api.ERR_UNSUPPORTED
    assert call(ok, 4, 0, o=FAKE + 16) == host_api.ERR_UNSUPPORTED   # 32-byte stores
    assert call(host_api.make_params(1, 64, 24, 2), 4, 0) == host_api.ERR_UNSUPPORTED
    assert call(host_api.make_params(1, 64, 32, 2, head_dim=64), 4, 0) == host_api.ERR_UNSUPPORTED
    assert call(host_api.make_params(0, 64, 32, 2), 4, 0, q=None) == host_api.OK   # nothing to do


@pytest.mark.parametrize("bad", ["dtype", "shape", "stride", "cpu"])
def test_window_attn_binding_refuses_wrong_tensors(bad):
    import torch
    p = host_api.make_params(1, 16, 4, 2)
    bf = torch.bfloat16
    Q, K = torch.zeros(1, 16, 4, 128, dtype=bf), torch.zeros(1, 16, 2, 128, dtype=bf)
    O, lse, V = torch.zeros_like(Q), torch.zeros(1, 4, 16), K.clone()
    if bad == "dtype":
        K = K.half()
    elif bad == "shape":
        V = V[:, :8].contiguous()
    elif bad == "stride":
        Q = torch.zeros(1, 4, 16, 128, dtype=bf).transpose(1, 2)
    with pytest.raises(host_api.InfLLMV2Error):
        host_api.window_attn(p, 4, 0, Q, K, V, O, lse)


def test_window_attn_binding_refuses_wrong_kinds():
    """What is no tensor, no 32-bit integer or another call's parameters."""
    import torch
    p, bf = host_api.make_params(1, 16, 4, 2), torch.bfloat16
    Q, K = torch.zeros(1, 16, 4, 128, dtype=bf), torch.zeros(1, 16, 2, 128, dtype=bf)
    rest = (Q, K, K, Q, torch.zeros(1, 4, 16))
    with pytest.raises(TypeError):
        host_api.window_attn(p, 4, 0, None, *rest[1:])
    with pytest.raises(TypeError):
        host_api.window_attn(p, 4.5, 0, *rest)
    with pytest.raises(OverflowError):
        host_api.window_attn(p, 1 << 31, 0, *rest)
    with pytest.raises(TypeError):
        host_api.window_attn(host_api.make_paged_params(1, 1, 1), 4, 0, *rest)
    with pytest.raises(TypeError):
        host_api.window_attn(None, 4, 0, *rest)
    with pytest.raises(host_api.InfLLMV2Error):   # tensors on the CPU
        host_api.window_attn(p, 4, 0, *rest)
