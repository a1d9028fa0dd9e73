"""GPU parity of the gated delta rule (prefill and cached step) against the
fp64 oracle on the same inputs.

Tolerances, set before the first run (u = 2^-24, the float32 half step):
  * float32 y and every state, token-by-token kernel: an update costs a handful
    of roundings (u each) and gates exact to a few 2^-22; the map
    a (I - beta k k^T) never lengthens a state row, so errors add up over the
    memory's horizon at worst: normwise 1e-5.
  * state of the chunked kernel: the same arithmetic in another order, with
    operands in two fp16 parts (2^-22 of a row's largest value dropped, at most),
    amplified by a chunk's triangular factor (its norm measured up to 8):
    normwise 8 * 2^-22 * sqrt(5 products) = 4.3e-6, and the tensor cores' own
    float32 sums: asserted at 1e-5 too.
  * bf16 y: the output rounding (half a step: 2^-8 of the value at worst, so at
    most 2^-8 / sqrt(3) = 2.3e-3 rms) and three operands rounded to one fp16
    part (2^-11 each): normwise 2.6e-3; elementwise 5 sigma of that against
    the head's rms: 1.3e-2 * max(rms, |ref|).
"""
import numpy as np
import pytest
import torch

import oracle
from selective_state_space_52_b200 import workloads as W

from gpu_util import Guarded

pytestmark = pytest.mark.gpu

SEQ = ("q", "k", "v", "dt_raw", "b_raw")


def close(got, ref, norm_tol, what, elem=None):
    got, ref = (np.asarray(t, dtype=np.float64) for t in (got, ref))
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.all(np.isfinite(got)), what + ": non-finite"
    rel = np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-30)
    assert rel <= norm_tol, f"{what}: normwise {rel:.3g}"
    rms = np.sqrt(np.mean(ref * ref)) if ref.size else 0.0
    off = np.abs(got - ref) / np.maximum(max(rms, 1e-30), np.abs(ref)) if ref.size else np.zeros(1)
    elem = 40 * norm_tol if elem is None else elem
    assert off.max() <= elem, f"{what}: an element is {off.max():.3g} off"


def tols(io):
    return (1e-5, None) if io == "f32" else (2.6e-3, 1.3e-2)


def make(N=128, P=128, G=2, H=4, io="bf16", L=130, B=2, seed=32):
    return W.make_delta_inputs(W.DeltaWorkload("t", B, L, G, H, seed, P, N, io))


def dev(inp):
    d = {k: v.cuda() for k, v in inp.items()}
    return d, {"dt_bias": d["dt_bias"], "A_log": d["A_log"]}


def run(inp, h0=True, lengths=None, in_place=False, **kw):
    from selective_state_space_52_b200 import axon_ssm
    d, params = dev(inp)
    B, L, H, P = d["v"].shape
    N = d["k"].shape[-1]
    gy, gh = Guarded((B, L, H, P), d["v"].dtype), Guarded((B, H, P, N), torch.float32)
    gy.t.fill_(7.0)
    h = d["h0"] if h0 else None
    if in_place:
        gh.t.copy_(h)
        h = gh.t
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    axon_ssm.delta_scan(*(d[k] for k in SEQ), params, h, lengths=ln, out=(gy.t, gh.t), **kw)
    torch.cuda.synchronize()
    assert gy.canaries_intact() and gh.canaries_intact()
    return gy.t.float().cpu().numpy(), gh.t.cpu().numpy()


def ref(inp, h0=True, lengths=None, qk_norm=True, scale=None):
    return oracle.delta_scan(*(inp[k] for k in SEQ), inp["dt_bias"], inp["A_log"], inp["h0"] if h0 else None,
                             lengths, scale, qk_norm)


def check(inp, what, state_tol=1e-5, **kw):
    y, h = run(inp, **kw)
    kw.pop("in_place", None)
    kw.pop("segments", None)
    y_ref, h_ref = ref(inp, **kw)
    io = "f32" if inp["v"].dtype == torch.float32 else "bf16"
    ln = kw.get("lengths")
    if ln is not None:
        for b, n in enumerate(ln):
            n = min(max(n, 0), y.shape[1])
            assert np.all(y[b, n:] == 7.0), f"{what}: y behind the end of row {b} was written"
            y_ref[b, n:] = 7.0
    if y.size:
        close(y, y_ref, tols(io)[0], what + " y", tols(io)[1])
    close(h, h_ref, state_tol, what + " state")


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 200, 333])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_lengths(cuda_lib, L, io):
    inp = make(L=L, io=io)
    check(inp, f"L{L} {io}")
    check(inp, f"L{L} {io} no h0", h0=False)
    if io == "bf16":
        check(inp, f"L{L} in chunks", segments=1)
        check(inp, f"L{L} in chunks, no h0", h0=False, segments=1)


@pytest.mark.parametrize("N, P", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("G, H", [(1, 1), (1, 3), (2, 2), (3, 12)])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_heads(cuda_lib, N, P, G, H, io):
    inp = make(N, P, G, H, io, L=100, B=1)
    check(inp, f"N{N} P{P} G{G} H{H} {io}")
    if io == "bf16":
        check(inp, f"N{N} P{P} G{G} H{H} in chunks", segments=1)


@pytest.mark.parametrize("segments", [0, 1, 2])
def test_raw_keys_and_queries(cuda_lib, segments):
    """Without the norm: keys of length 1/4 to 4 with beta |k|^2 up to 1.6, queries
    from 1e-6 to 1e6 long within one chunk; tokens are compared each by its size."""
    inp = make(L=200, B=1, G=2, H=4)
    k, q = inp["k"].float(), inp["q"].float()
    size = 4.0 ** torch.linspace(-1, 1, 200)[torch.randperm(200, generator=torch.Generator().manual_seed(3))]
    inp["k"] = (k / k.norm(dim=-1, keepdim=True) * size[None, :, None, None]).bfloat16()
    inp["b_raw"] = torch.full_like(inp["b_raw"], -2.2)                          # beta = 0.1
    far = 10.0 ** (torch.arange(200) % 13 - 6)
    inp["q"] = (q / q.norm(dim=-1, keepdim=True) * far[None, :, None, None]).bfloat16()
    y, h = run(inp, segments=segments, qk_norm=False)
    y_ref, h_ref = ref(inp, qk_norm=False)
    f = far.numpy()[None, :, None, None]
    close(y / f, y_ref / f, 2.6e-3, "y", 1.3e-2)
    close(h, h_ref, 1e-5, "state")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_many_blocks(cuda_lib, io):
    """Enough heads that every block keeps the most rows a lane holds."""
    check(make(G=16, H=32, B=5, L=70, io=io), "B5 H32 " + io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [dict(qk_norm=False), dict(scale=1.0), dict(scale=-0.3, qk_norm=False)])
def test_norm_and_scale(cuda_lib, io, kw):
    inp = make(L=150, io=io)
    if not kw.get("qk_norm", True):
        for n in ("q", "k"):
            t = inp[n].float()
            inp[n] = (t / t.norm(dim=-1, keepdim=True)).to(inp[n].dtype)
    check(inp, str(kw), **kw)


@pytest.mark.parametrize("io, segments", [("bf16", 0), ("bf16", 1), ("bf16", 3), ("f32", 0)])
def test_ragged_rows(cuda_lib, io, segments):
    """Rows of every kind of length; what lies behind a row's end is NaN and
    infinity, and y there stays as it was."""
    lengths = [0, 1, 63, 64, 65, 130, 150, 400, -3]                 # the last two are taken into 0 .. L
    inp = make(B=len(lengths), L=150, io=io)
    dirty = {k: v.clone() for k, v in inp.items()}
    for b, n in enumerate(lengths):
        n = min(max(n, 0), 150)
        for i, name in enumerate(SEQ):
            dirty[name][b, n:] = (float("nan"), float("inf"), -float("inf"))[i % 3]
            inp[name][b, n:] = 0
    y, h = run(dirty, lengths=lengths, segments=segments)
    y_ref, h_ref = ref(inp, lengths=lengths)
    for b, n in enumerate(lengths):
        n = min(max(n, 0), 150)
        assert np.all(y[b, n:] == 7.0), b
        if n:
            close(y[b, :n], y_ref[b, :n], tols(io)[0], f"y of row {b}", tols(io)[1])
        close(h[b], h_ref[b], 1e-5, f"state of row {b}")
        if n == 0:
            np.testing.assert_array_equal(h[b], inp["h0"][b].numpy())


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("L", [0, 40, 300])
def test_state_in_place(cuda_lib, io, L):
    check(make(L=L, io=io), f"in place L{L}", in_place=True)
    if io == "bf16" and L:
        for segments in (1, 3):
            check(make(L=L, io=io), f"in place L{L}, {segments} segments", in_place=True, segments=segments)


@pytest.mark.parametrize("L, segments", [(40, 0), (40, 1), (300, 0), (300, 2)])
def test_slices_of_one_projection(cuda_lib, L, segments):
    """q, k and v as slices of one row (tokens at the row's stride), bit for
    bit what dense tensors give."""
    from selective_state_space_52_b200 import axon_ssm
    d, params = dev(make(L=L, B=2, G=2, H=4))
    rowed = torch.cat([torch.full((2, L, 8), float("nan"), device="cuda", dtype=torch.bfloat16)] +
                      [d[n].flatten(2) for n in ("q", "k", "v")] +
                      [torch.full((2, L, 24), float("nan"), device="cuda", dtype=torch.bfloat16)], dim=-1)
    q = rowed[..., 8:264].unflatten(-1, (2, 128))
    k = rowed[..., 264:520].unflatten(-1, (2, 128))
    v = rowed[..., 520:1032].unflatten(-1, (4, 128))
    y, h = axon_ssm.delta_scan(*(d[n] for n in SEQ), params, d["h0"], segments=segments)
    y2, h2 = axon_ssm.delta_scan(q, k, v, d["dt_raw"], d["b_raw"], params, d["h0"], segments=segments)
    assert torch.equal(y, y2) and torch.equal(h, h2)


def extreme(io, L=200):
    """Head 0 forgets nothing (dt underflows to a decay of 1), head 1 forgets
    all (decay 0 within a token), head 2 writes nothing (beta 0), head 3 takes
    one large jump in a slow decay; keys of both key heads partly repeated, a
    zero key and a zero query among them."""
    inp = make(io=io, L=L, B=1)
    inp["dt_bias"][:] = torch.tensor([-60.0, 80.0, -3.0, -6.0])
    inp["A_log"][:] = torch.tensor([0.0, 2.7, 1.0, 0.0])
    inp["b_raw"][:, :, 2] = -200.0
    inp["b_raw"][:, 50:60] = 90.0
    inp["dt_raw"][:, 100, 3] = 300.0
    inp["k"][:, 20:90] = inp["k"][:, 20:21]
    inp["k"][:, 130] = 0.0
    inp["q"][:, 131] = 0.0
    return inp


@pytest.mark.parametrize("io, segments", [("bf16", 0), ("bf16", 1), ("bf16", 2), ("f32", 0)])
def test_extreme_gates(cuda_lib, io, segments):
    inp = extreme(io)
    y, h = run(inp, segments=segments)
    y_ref, h_ref = ref(inp)
    for hd in range(4):
        close(y[:, :, hd], y_ref[:, :, hd], tols(io)[0], f"y of head {hd}", tols(io)[1])
        close(h[:, hd], h_ref[:, hd], 1e-5, f"state of head {hd}")


@pytest.mark.parametrize("io, segments", [("bf16", 0), ("bf16", 1), ("bf16", 2), ("f32", 0)])
def test_infinite_gates(cuda_lib, io, segments):
    """dt_raw of +inf forgets everything, -inf nothing; b_raw likewise."""
    inp = make(io=io, L=70, B=1)
    want = {k: v.clone() for k, v in inp.items()}
    for name, t, big in (("dt_raw", 10, 3e4), ("dt_raw", 20, -3e4), ("b_raw", 30, 3e4), ("b_raw", 40, -3e4)):
        inp[name][:, t] = float("inf") if big > 0 else -float("inf")
        want[name][:, t] = big
    y, h = run(inp, segments=segments)
    y_ref, h_ref = ref(want)
    close(y, y_ref, tols(io)[0], "y", tols(io)[1])
    close(h, h_ref, 1e-5, "state")


@pytest.mark.parametrize("segments", [0, 1, 2])
def test_nan_gate_shows(cuda_lib, segments):
    """A NaN in a gate is not swallowed: its head's later outputs are NaN, the others' are not."""
    inp = make(L=90, B=1)
    inp["dt_raw"][0, 10, 1] = float("nan")
    y, h = run(inp, segments=segments)
    assert np.isnan(y[0, 64:, 1]).all() and np.isnan(h[0, 1]).all()
    assert np.isfinite(y[0, :, [0, 2, 3]]).all() and np.isfinite(h[0, [0, 2, 3]]).all()


@pytest.mark.parametrize("name", ["A_log", "dt_bias"])
@pytest.mark.parametrize("segments", [0, 1, 2])
def test_nan_parameter_shows(cuda_lib, segments, name):
    """A NaN parameter reaches its head's outputs and state (the scan's and the step's), no other's."""
    from selective_state_space_52_b200 import axon_ssm
    inp = make(L=90, B=1)
    inp[name][1] = float("nan")
    y, h = run(inp, segments=segments)
    assert np.isnan(y[0, 1:, 1]).all() and np.isnan(h[0, 1]).all()
    assert np.isfinite(y[0, :, [0, 2, 3]]).all() and np.isfinite(h[0, [0, 2, 3]]).all()
    d, params = dev(inp)
    state = torch.ones_like(d["h0"])
    y1 = axon_ssm.delta_step(*(d[n][:, 0] for n in SEQ[:3]), *(d[n][:, 0].contiguous() for n in SEQ[3:]), params, state)
    assert y1[0, 1].isnan().all() and state[0, 1].isnan().all()
    assert y1[0, [0, 2, 3]].isfinite().all() and state[0, [0, 2, 3]].isfinite().all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_two_calls_and_streams_agree(cuda_lib, io):
    """Back-to-back calls on one workspace, a call on another stream and a
    captured graph replayed twice: bit for bit the same."""
    from selective_state_space_52_b200 import axon_ssm
    d, params = dev(make(L=300, io=io))
    other, _ = dev(make(L=300, io=io, seed=77))
    B, L, H, P = d["v"].shape
    io_code = axon_ssm.AXON_F32 if io == "f32" else axon_ssm.AXON_BF16
    ws = torch.empty(max(16, axon_ssm.axon_delta_workspace_bytes(B, L, H, 2, P, 128, io_code)), dtype=torch.uint8, device="cuda")
    y, h = axon_ssm.delta_scan(*(d[n] for n in SEQ), params, d["h0"], workspace=ws)
    axon_ssm.delta_scan(*(other[n] for n in SEQ), params, other["h0"], workspace=ws, check=False)
    y2, h2 = axon_ssm.delta_scan(*(d[n] for n in SEQ), params, d["h0"], workspace=ws)
    assert torch.equal(y, y2) and torch.equal(h, h2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y3, h3 = axon_ssm.delta_scan(*(d[n] for n in SEQ), params, d["h0"], stream=side, check=False)
    side.synchronize()
    assert torch.equal(y, y3) and torch.equal(h, h3)
    out = torch.zeros_like(y), torch.zeros_like(h)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        axon_ssm.delta_scan(*(d[n] for n in SEQ), params, d["h0"], workspace=ws, out=out, check=False)
    for _ in range(2):
        out[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, out[0]) and torch.equal(h, out[1])


# ------------------------------------------------------------ chunks and segments
@pytest.mark.parametrize("segments", [1, 2, 3, 4, 7, 64])
@pytest.mark.parametrize("N, P", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_segments(cuda_lib, segments, N, P):
    """Any cut of the sequence (7 chunks, the last ragged) gives the same answer."""
    check(make(N, P, 2, 4, L=430, B=1), f"{segments} segments, N{N} P{P}", segments=segments)


@pytest.mark.parametrize("segments", [2, 3, 7])
def test_segments_of_ragged_rows(cuda_lib, segments):
    """Rows that end in every segment, before a segment's first token and at its
    last, and a row of no tokens; the state in place."""
    lengths = [0, 1, 64, 65, 128, 190, 192, 193, 320, 430]
    inp = make(G=1, H=2, B=len(lengths), L=430)
    check(inp, f"{segments} segments", segments=segments, lengths=lengths)
    check(inp, f"{segments} segments in place", segments=segments, lengths=lengths, in_place=True)


def test_no_rows_and_wrong_types(cuda_lib):
    from selective_state_space_52_b200 import axon_ssm
    d, params = dev(make(L=70, B=2))
    none = [d[n][:0] for n in SEQ]
    y, h = axon_ssm.delta_scan(*none, params)
    assert y.shape == (0, 70, 4, 128) and h.shape == (0, 4, 128, 128)
    assert axon_ssm.delta_step(*(t[:, 0] for t in none[:3]), *(t[:, 0].contiguous() for t in none[3:]), params,
                               d["h0"][:0]).shape == (0, 4, 128)
    seq = [d[n] for n in SEQ]
    bad = [
        (TypeError, lambda: axon_ssm.delta_scan(*(t.half() for t in seq), params)),
        (TypeError, lambda: axon_ssm.delta_scan(seq[0].float(), *seq[1:], params)),
        (TypeError, lambda: axon_ssm.delta_scan(*seq, params, d["h0"].bfloat16())),
        (TypeError, lambda: axon_ssm.delta_scan(*seq, params, lengths=torch.tensor([3, 4], device="cuda"))),
        (ValueError, lambda: axon_ssm.delta_scan(*seq, params, lengths=torch.tensor([3, 4], dtype=torch.int32))),
        (ValueError, lambda: axon_ssm.delta_scan(seq[0][:, :-1], *seq[1:], params)),
        (ValueError, lambda: axon_ssm.delta_scan(seq[0][..., ::2], seq[1][..., ::2], *seq[2:], params)),
        (ValueError, lambda: axon_ssm.delta_scan(*seq[:3], seq[3].transpose(0, 1).contiguous().transpose(0, 1), seq[4], params)),
        (ValueError, lambda: axon_ssm.delta_scan(*seq, params, d["h0"][:, :, :, ::2])),
        (axon_ssm.AxonError, lambda: axon_ssm.delta_scan(*seq, params, segments=-1)),
        (axon_ssm.AxonError, lambda: axon_ssm.delta_scan(*seq, params, segments=1, workspace=torch.empty(512, dtype=torch.uint8, device="cuda"))),
        (axon_ssm.AxonError, lambda: axon_ssm.delta_scan(*seq, params, out=(d["v"], torch.empty_like(d["h0"])))),
        (axon_ssm.AxonError, lambda: axon_ssm.delta_scan(*seq, params, scale=float("nan"))),
        (ValueError, lambda: axon_ssm.delta_step(*(t[:, 0] for t in seq[:3]), seq[3][:, 0], seq[4][:, 0], params, d["h0"][:1])),
        (ValueError, lambda: axon_ssm.gated_norm(d["v"], torch.ones(3, device="cuda"))),
        (ValueError, lambda: axon_ssm.gated_norm(d["v"], z=d["v"][:1])),
        (TypeError, lambda: axon_ssm.gated_norm(d["v"], z=d["v"].float())),
        (axon_ssm.AxonError, lambda: axon_ssm.gated_norm(d["v"], group=96)),
        (KeyError, lambda: axon_ssm.gated_norm(d["v"], kind="layer")),
    ]
    for n, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            pytest.fail(f"call {n} went through")


def test_given_workspaces(cuda_lib):
    """Of any type; on the inputs' device or refused."""
    from selective_state_space_52_b200 import axon_ssm
    d, params = dev(make(L=130, B=1))
    seq = [d[n] for n in SEQ]
    n = axon_ssm.axon_delta_workspace_bytes(1, 130, 4, 2, 128, 128, axon_ssm.AXON_BF16, 1)
    want = axon_ssm.delta_scan(*seq, params, segments=1)
    for dtype in (torch.uint8, torch.float32, torch.int64):
        ws = torch.empty((2, n // 2 // dtype.itemsize), dtype=dtype, device="cuda")
        got = axon_ssm.delta_scan(*seq, params, segments=1, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert axon_ssm.delta_error_flag(ws) == 0
    with pytest.raises(ValueError):
        axon_ssm.delta_scan(*seq, params, segments=1, workspace=torch.empty(n, dtype=torch.uint8))


def test_error_flag_stays_clear(cuda_lib):
    from selective_state_space_52_b200 import axon_ssm
    d, params = dev(make(L=300, B=1))
    for segments in (1, 3):
        n = axon_ssm.axon_delta_workspace_bytes(1, 300, 4, 2, 128, 128, axon_ssm.AXON_BF16, segments)
        ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")        # a nonzero flag beforehand, garbage in the rest
        y, h = axon_ssm.delta_scan(*(d[k] for k in SEQ), params, d["h0"], workspace=ws, segments=segments)
        assert axon_ssm.delta_error_flag(ws) == 0
        assert torch.isfinite(y).all() and torch.isfinite(h).all()


@pytest.mark.parametrize("segments", [1, 3])
@pytest.mark.parametrize("power", [-60, -20, 20, 60])
def test_scaled_values(cuda_lib, power, segments):
    """Everything is linear in v and h0: values of any size, through the lanes' scales."""
    inp = make(L=300, B=1)
    inp["v"] = (inp["v"].float() * 2.0 ** power).bfloat16()
    inp["h0"] = inp["h0"] * 2.0 ** power
    check(inp, f"values times 2^{power}", segments=segments)


@pytest.mark.parametrize("segments", [1, 3])
def test_outliers_in_v(cuda_lib, segments):
    """Columns of very different size, and single values far above the rest of
    their column, so that lanes rescale on the way; each size is checked by itself."""
    inp = make(L=400, B=1, H=2, G=1)
    size = torch.logspace(-6, 6, 128)
    inp["v"] = (inp["v"].float() * size).bfloat16()
    inp["v"][0, 100, :, ::7] = (1e5 * size[::7]).bfloat16()
    inp["v"][0, 101, :, 3::11] = 0
    inp["h0"] = inp["h0"] * size[:, None]
    y, h = run(inp, segments=segments)
    y_ref, h_ref = ref(inp)
    for v in range(0, 128, 5):
        close(y[..., v], y_ref[..., v], 2.6e-3, f"y of column {v}", 2e-2)
        close(h[:, :, v], h_ref[:, :, v], 1e-5, f"state of column {v}")


@pytest.mark.parametrize("segments", [0, 1, 3])
def test_silent_stretch(cuda_lib, segments):
    """No values for 200 tokens: the state only decays and forgets what the keys
    touch.  A lane's numbers are kept to 2^-21 of its largest at the start of a
    chunk, and 21 chunks' worth of such errors stay below 1e-5 of the state
    before the stretch (nothing brings them up: the map never lengthens a row)."""
    inp = make(L=200, B=1)
    inp["v"][:] = 0
    y, h = run(inp, segments=segments)
    y_ref, h_ref = ref(inp)
    assert np.abs(h - h_ref).max() <= 1e-5 * np.abs(inp["h0"].numpy()).max()
    close(y, y_ref, 2.6e-3, "y", 1.3e-2)


def test_long_offsets(cuda_lib):
    """2^31 values of v and of y: the last head of the wide call, bit for bit what
    a call on that head alone gives (it reads the same tensors at their strides)."""
    from selective_state_space_52_b200 import axon_ssm
    L, H, P, N = 131072, 128, 128, 64
    g = torch.Generator(device="cuda").manual_seed(9)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)

    q, k, v = normal(1, L, 1, N), normal(1, L, 1, N), normal(1, L, H, P)
    dt_raw, b_raw = normal(1, L, H), normal(1, L, H)
    params = {"dt_bias": torch.full((H,), -4.0, device="cuda"), "A_log": torch.linspace(0, 2, H, device="cuda")}
    y, h = axon_ssm.delta_scan(q, k, v, dt_raw, b_raw, params, segments=1)
    one = {n: t[-1:].clone() for n, t in params.items()}
    y1, h1 = axon_ssm.delta_scan(q, k, v[:, :, -1:], dt_raw[..., -1:].contiguous(), b_raw[..., -1:].contiguous(), one, segments=1)
    assert torch.equal(y[:, :, -1:], y1) and torch.equal(h[:, -1:], h1)
    assert torch.isfinite(y1).all() and float(y1[:, -1].float().abs().max()) > 0


# ------------------------------------------------------------ the cached step
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N, P", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("B, G, H", [(1, 1, 1), (3, 2, 6), (40, 4, 16)])
def test_step(cuda_lib, io, N, P, B, G, H):
    from selective_state_space_52_b200 import axon_ssm
    inp = make(N, P, G, H, io, L=1, B=B)
    d, params = dev(inp)
    st = Guarded((B, H, P, N), torch.float32, fill=d["h0"])
    gy = Guarded((B, H, P), d["v"].dtype)
    axon_ssm.delta_step(*(d[n][:, 0] for n in ("q", "k", "v")), *(d[n][:, 0].contiguous() for n in ("dt_raw", "b_raw")),
                        params, st.t, y=gy.t)
    torch.cuda.synchronize()
    assert st.canaries_intact() and gy.canaries_intact()
    y_ref, h_ref = ref(inp)
    close(gy.t.float().cpu().numpy(), y_ref[:, 0], tols(io)[0], "y", tols(io)[1])
    close(st.t.cpu().numpy(), h_ref, 1e-5, "state")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_step_extremes(cuda_lib, io):
    from selective_state_space_52_b200 import axon_ssm
    inp = extreme(io)
    for t in (0, 55, 100, 130, 131):
        one = {k: (v[:, t:t + 1].contiguous() if k in SEQ else v) for k, v in inp.items()}
        d, params = dev(one)
        y = axon_ssm.delta_step(*(d[n][:, 0] for n in SEQ), params, d["h0"], qk_norm=False, scale=0.5)
        y_ref, h_ref = ref(one, qk_norm=False, scale=0.5)
        close(y.float().cpu().numpy(), y_ref[:, 0], tols(io)[0], f"y of token {t}", tols(io)[1])
        close(d["h0"].cpu().numpy(), h_ref, 1e-5, f"state after token {t}")


# ------------------------------------------------------------ together, as a program uses them
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_prefill_then_decode_then_norm(cuda_lib, io):
    """A prompt in two pieces (the second continues the first), six decode
    steps, the output norm with its gate on every token: against the oracle's
    one run over the whole sequence."""
    from selective_state_space_52_b200 import axon_ssm
    L, cut, steps = 150, 83, 6
    inp = make(L=L + steps, io=io)
    d, params = dev(inp)
    dt = d["v"].dtype
    B, _, H, P = d["v"].shape
    g = torch.Generator().manual_seed(5)
    z = torch.randn(B, L + steps, H * P, generator=g).to(dt)
    w = 1 + 0.1 * torch.randn(P, generator=g)
    zc, wc = z.cuda(), w.cuda()
    ys, h = [], d["h0"]
    for a, b in ((0, cut), (cut, L)):
        y, h = axon_ssm.delta_scan(*(d[n][:, a:b].contiguous() for n in SEQ), params, h)
        ys.append(axon_ssm.gated_norm(y.flatten(2), wc, zc[:, a:b].contiguous(), group=P))
    for t in range(L, L + steps):
        y = axon_ssm.delta_step(*(d[n][:, t].contiguous() for n in SEQ), params, h)
        ys.append(axon_ssm.gated_norm(y.flatten(1), wc, zc[:, t], group=P)[:, None])
    got = torch.cat(ys, 1).float().cpu().numpy()
    y_ref, h_ref = ref(inp)
    o_ref = oracle.gated_norm(y_ref.reshape(B, L + steps, H * P), P, "rms", "after", True, z, w)
    # the norm sees y rounded to the io type, and rounds once more
    close(got, o_ref, 1e-5 if io == "f32" else 2.6e-3 + 2.3e-3, "normed output", None if io == "f32" else 4e-2)
    close(h.cpu().numpy(), h_ref, 1e-5, "state")


@pytest.mark.parametrize("L", [20, 200])
def test_captured_run_replays(cuda_lib, L):
    """Prefill, norm and a step in one captured graph, replayed on other values: as eager calls."""
    from selective_state_space_52_b200 import axon_ssm
    a, params = dev(make(L=L, B=2))
    b = dev(make(L=L, B=2, seed=33))[0]
    w = torch.rand(128, device="cuda") + 0.5

    def calls(d):
        y, h = axon_ssm.delta_scan(*(d[n] for n in SEQ), params, d["h0"], check=False)
        o = axon_ssm.gated_norm(y.flatten(2), w, d["v"].flatten(2), group=128)
        y1 = axon_ssm.delta_step(*(d[n][:, 3].contiguous() for n in SEQ), params, h)
        return y, h, o, y1

    want = [t.clone() for t in calls(b)]
    graph = torch.cuda.CUDAGraph()
    calls(a)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = calls(a)
    for n in (*SEQ, "h0"):
        a[n].copy_(b[n])
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("io, segments", [("bf16", 0), ("bf16", 1), ("bf16", 2), ("f32", 0)])
def test_zero_keys_queries_and_values(cuda_lib, io, segments):
    """Tokens whose key, query or value is 0: the norm's eps keeps them finite."""
    inp = make(io=io, L=130, B=1)
    inp["k"][:, 3:60:5] = 0
    inp["q"][:, 2:130:7] = 0
    inp["v"][:, 64:128] = 0
    y, h = run(inp, segments=segments)
    y_ref, h_ref = ref(inp)
    assert (y[:, 2:130:7] == 0).all()
    close(y, y_ref, tols(io)[0], "y", tols(io)[1])
    close(h, h_ref, 1e-5, "state")


# ------------------------------------------------------------ y: two parts an operand, one rounding
@pytest.mark.parametrize("segments", [1, 3])
@pytest.mark.parametrize("N, P", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_y_is_rounded_once(cuda_lib, N, P, segments):
    """y in chunks is the exact value rounded to bf16, not a value some 2^-11
    off that is then rounded.  With both parts of S, U and M in its products
    the value before the rounding is within 4e-6 of its head's rms (as the
    state: 2^-21 an operand, five products, the factor's amplification).

    * Equal to the rounded oracle: a value y changes sides with probability
      |err| / step, step >= 2^-8 |y|, so over normal values of rms 1 at most
      0.8 d (1 + ln(1 / d)) with d = 4e-6 * 2^8 = 1e-3: 0.7%.  Asserted: 1%.
    * No bias: the slope of y on the oracle's y is 1 to six sigma of the
      rounding's own noise, 2^-8 / sqrt(3) sqrt(sum r^4) / sum r^2, and the
      curvature of the values' density over a step, (2^-7)^2 / 12 < 2^-17.
    """
    inp = make(N, P, 2, 4, L=1000, B=1)
    y, _ = run(inp, segments=segments)
    y_ref, _ = ref(inp)
    want = torch.from_numpy(y_ref).bfloat16().float().numpy()
    assert np.mean(y != want) <= 0.01, np.mean(y != want)
    s2 = np.sum(y_ref ** 2)
    slope = np.sum(y * y_ref) / s2
    noise = 2 ** -8 / np.sqrt(3) * np.sqrt(np.sum(y_ref ** 4)) / s2
    assert abs(slope - 1) <= 6 * noise + 2 ** -17, (slope - 1, noise)


# ------------------------------------------------------------ values anywhere in float32's range
@pytest.mark.parametrize("segments", [1, 3])
@pytest.mark.parametrize("power", [-110, -90, 90, 115])
def test_values_near_the_types_limits(cuda_lib, power, segments):
    """As test_scaled_values, up to where a state of some 2^8 times the values is still finite
    (and down to where few of its elements leave the normal range)."""
    inp = make(L=300, B=1)
    inp["v"] = (inp["v"].double() * 2.0 ** power).bfloat16()
    inp["h0"] = (inp["h0"].double() * 2.0 ** power).float()
    y, h = run(inp, segments=segments)
    y_ref, h_ref = ref(inp)
    close(y / 2.0 ** power, y_ref / 2.0 ** power, 2.6e-3, "y", 1.3e-2)
    close(h / 2.0 ** power, h_ref / 2.0 ** power, 1e-5, "state")


@pytest.mark.parametrize("segments", [0, 1, 3])
@pytest.mark.parametrize("first, then", [(-70, 70), (-110, 20), (0, 110), (110, -5), (70, -70)])
def test_values_jump(cuda_lib, first, then, segments):
    """Values of one size, then, from a chunk on, of another: up by 2^110 or 2^140 at once,
    or down, after a decay that leaves nothing of the first."""
    inp = make(L=330, B=1)
    v = inp["v"].double()
    v[:, :192] *= 2.0 ** first
    v[:, 192:] *= 2.0 ** then
    inp["h0"] = inp["h0"] * 0
    if first > then:
        v[:, 150:192] = 0
        inp["dt_raw"][:, 150:160] = 60.0             # e^-60 at most, at each of ten tokens
    inp["v"] = v.bfloat16()
    y, h = run(inp, segments=segments)
    y_ref, h_ref = ref(inp)
    for a, b, p in ((0, 192, first), (192, 330, then)):
        close(y[:, a:b] / 2.0 ** p, y_ref[:, a:b] / 2.0 ** p, 2.6e-3, f"y of tokens {a} to {b}", 1.3e-2)
    close(h / 2.0 ** then, h_ref / 2.0 ** then, 1e-5, "state")


@pytest.mark.parametrize("segments", [0, 1, 2])
@pytest.mark.parametrize("power", [-110, 110, 118])
def test_raw_queries_of_any_length(cuda_lib, power, segments):
    """Without the norm: queries 2^power long, values that bring y back to normal size."""
    inp = make(L=200, B=1)
    k, q = inp["k"].float(), inp["q"].double()
    inp["k"] = (k / k.norm(dim=-1, keepdim=True)).bfloat16()
    inp["q"] = (q / q.norm(dim=-1, keepdim=True) * 2.0 ** power).bfloat16()
    inp["v"] = (inp["v"].double() * 2.0 ** (-power // 2)).bfloat16()
    inp["h0"] = (inp["h0"].double() * 2.0 ** (-power // 2)).float()
    y, h = run(inp, segments=segments, qk_norm=False)
    y_ref, h_ref = ref(inp, qk_norm=False)
    p = 2.0 ** (power - power // 2)
    close(y / p, y_ref / p, 2.6e-3, "y", 1.3e-2)
    close(h / 2.0 ** (-power // 2), h_ref / 2.0 ** (-power // 2), 1e-5, "state")


# ------------------------------------------------------------ raw keys too long for the chunks
def long_keys(what, L=200):
    inp = make(L=L, B=1)
    for n in ("q", "k"):
        t = inp[n].float()
        inp[n] = (t / t.norm(dim=-1, keepdim=True)).bfloat16()
    k = inp["k"].float()
    if what == "growing":            # beta |k|^2 = 4 along one key: the state's part grows by 3 a token, 3^20 in all
        k[:, 70:90] = 2 * k[:, 70:71]
        inp["b_raw"][:, 70:90] = 90.0
        inp["dt_bias"][:] = -60.0
    elif what == "long":             # one key of 2^20, hardly taken up
        k[:, 100] *= 2.0 ** 20
        inp["b_raw"][:, 100] = -30.0
    elif what == "last token":       # one of the padded last chunk
        k[:, -1] *= 2.0 ** 20
    inp["k"] = k.bfloat16()
    return inp


@pytest.mark.parametrize("segments", [1, 3])
@pytest.mark.parametrize("what", ["growing", "long", "last token"])
def test_keys_too_long_are_reported(cuda_lib, what, segments):
    from selective_state_space_52_b200 import axon_ssm
    inp = long_keys(what)
    d, params = dev(inp)
    with pytest.raises(axon_ssm.AxonError) as e:
        axon_ssm.delta_scan(*(d[n] for n in SEQ), params, d["h0"], qk_norm=False, segments=segments)
    assert e.value.status == 2
    ws = torch.empty(axon_ssm.axon_delta_workspace_bytes(1, 200, 4, 2, 128, 128, axon_ssm.AXON_BF16, segments),
                     dtype=torch.uint8, device="cuda")
    axon_ssm.delta_scan(*(d[n] for n in SEQ), params, d["h0"], qk_norm=False, segments=segments, workspace=ws, check=False)
    assert axon_ssm.delta_error_flag(ws) == 2
    # the same workspace afterwards: the flag is cleared, and normalised keys may be of any length
    y, h = axon_ssm.delta_scan(*(d[n] for n in SEQ), params, d["h0"], segments=segments, workspace=ws)
    assert axon_ssm.delta_error_flag(ws) == 0
    y_ref, h_ref = ref(inp)
    close(y.float().cpu().numpy(), y_ref, 2.6e-3, "y", 1.3e-2)
    close(h.cpu().numpy(), h_ref, 1e-5, "state")


@pytest.mark.parametrize("segments", [1, 3])
@pytest.mark.parametrize("ragged", [False, True])
def test_nan_with_raw_keys_is_no_error(cuda_lib, segments, ragged):
    """A NaN or infinity among the inputs comes out as one and is not reported as keys too
    long; one behind a row's end is no excuse for keys that are."""
    from selective_state_space_52_b200 import axon_ssm
    inp = long_keys("none")
    inp["v"][0, 70, 1, 5] = float("nan")
    inp["v"][0, 70, 1, 6] = float("inf")
    inp["dt_raw"][0, 90, 2] = float("nan")
    kw = dict(lengths=[190]) if ragged else {}
    n = 190 if ragged else 200
    y, h = run(inp, qk_norm=False, segments=segments, **kw)
    for col in (5, 6):
        assert not np.isfinite(y[0, 128:n, 1, col]).any() and not np.isfinite(h[0, 1, col]).any()
    assert np.isnan(y[0, 128:n, 2]).all() and np.isnan(h[0, 2]).all()
    assert np.isfinite(y[0, :, [0, 3]]).all() and np.isfinite(h[0, [0, 3]]).all()
    if ragged:
        inp = long_keys("long")
        inp["v"][0, 195] = float("nan")
        with pytest.raises(axon_ssm.AxonError):
            run(inp, qk_norm=False, segments=segments, **kw)


def test_keys_too_long_token_by_token(cuda_lib):
    """The float32 kernel has no such limit."""
    inp = {n: t.float() if n in SEQ else t for n, t in long_keys("long").items()}
    y, h = run(inp, qk_norm=False)
    y_ref, h_ref = ref(inp, qk_norm=False)
    close(y, y_ref, 1e-5, "y")
    close(h, h_ref, 1e-5, "state")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("H", [1, 3, 4])
def test_rates_at_any_token(cuda_lib, io, H):
    """One sequence's rates of any token, and parameters out of a longer array: contiguous, aligned only to a value."""
    from selective_state_space_52_b200 import axon_ssm
    L = 70
    inp = make(G=1, H=H, io=io, L=L, B=1)
    d, params = dev(inp)
    params = {n: torch.cat([t.new_zeros(1), t])[1:] for n, t in params.items()}
    state = d["h0"].clone()
    y_ref, h_ref = ref(inp)
    ys = [axon_ssm.delta_step(*(d[n][:, t] for n in SEQ), params, state) for t in range(3)]
    y, h = axon_ssm.delta_scan(*(d[n][:, 3:] for n in SEQ), params, state)
    ys = torch.cat([*(t[:, None] for t in ys), y], 1).float().cpu().numpy()
    close(ys, y_ref, tols(io)[0], "y", tols(io)[1])
    close(h.cpu().numpy(), h_ref, 1e-5, "state")
    if io == "bf16":
        y, h = axon_ssm.delta_scan(*(d[n][:, 3:] for n in SEQ), params, state, segments=1)
        close(y.float().cpu().numpy(), y_ref[:, 3:], 2.6e-3, "y in chunks", 1.3e-2)
        close(h.cpu().numpy(), h_ref, 1e-5, "state in chunks")


# ------------------------------------------------------------ long sequences, cut as long prompts are
@pytest.mark.parametrize("N, P", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_long_segments_after_a_fold(cuda_lib, N, P):
    """21 chunks in three segments of seven: the last enters with a fold and then goes
    more than twice round the three stages that held the transitions."""
    check(make(N, P, 1, 2, L=1300, B=1), f"three segments, N{N} P{P}", segments=3)


@pytest.mark.parametrize("segments", [3, 4])
def test_long_segments_of_ragged_rows(cuda_lib, segments):
    """Rows that end in every segment and at a segment's and a chunk's end, in place and without a state."""
    lengths = [1300, 1299, 1090, 897, 896, 500, 448, 64, 0]
    inp = make(G=1, H=2, B=len(lengths), L=1300)
    check(inp, f"{segments} segments in place", segments=segments, lengths=lengths, in_place=True)
    check(inp, f"{segments} segments, no h0", segments=segments, lengths=lengths, h0=False)


@pytest.mark.parametrize("segments", [0, 1, 3, 8])
def test_long_memory(cuda_lib, segments):
    """4096 tokens whose decays keep some thousand of them; segments = 0 cuts the sequence.
    A chunk's error is 2^-22 an operand and five products, of either sign over the
    64 chunks: sqrt(64 * 5) 2^-22 = 4.3e-6, asserted as everywhere at 1e-5."""
    from selective_state_space_52_b200 import axon_ssm
    inp = make(G=1, H=2, L=4096, B=1)
    inp["dt_bias"][:] = torch.tensor([-7.0, -8.0])
    inp["A_log"][:] = 0.0
    if segments == 0:
        size = lambda s: axon_ssm.axon_delta_workspace_bytes(1, 4096, 2, 1, 128, 128, axon_ssm.AXON_BF16, s)    # noqa: E731
        assert size(0) > size(1)
    check(inp, "long memory", segments=segments)


def test_cut_by_the_library(cuda_lib):
    """One chunk short of a full cut, few heads: the library's own segments."""
    from selective_state_space_52_b200 import axon_ssm
    size = lambda s: axon_ssm.axon_delta_workspace_bytes(2, 2047, 2, 1, 128, 64, axon_ssm.AXON_BF16, s)      # noqa: E731
    assert size(0) > size(1)
    check(make(128, 64, 1, 2, L=2047, B=2), "the library's segments", lengths=[2047, 1111])


def test_wait_gives_up_and_reports(cuda_lib):
    """The walk's failure path: a wait that nothing ends gives up, the block's other waits
    end with it, the flag is set, products are drained and the tensor memory is freed, so
    that the chunked kernels (which need all of an SM's) run as before afterwards."""
    from selective_state_space_52_b200 import axon_ssm
    for limit in (1, 64, 3000):
        status = torch.full((2,), -1, dtype=torch.int32, device="cuda")
        axon_ssm.axon_delta_wait_probe(status, limit)
        torch.cuda.synchronize()
        assert status.tolist() == [7, 1], limit
    check(make(G=16, H=32, B=5, L=100), "after the probe", segments=1)


# ------------------------------------------------------------ tokens that hardly write
@pytest.mark.parametrize("segments", [1, 3])
@pytest.mark.parametrize("gate", [-5.0, -8.0, -12.0, -20.0, -60.0])
@pytest.mark.parametrize("N, P", [(64, 128), (128, 64)])
def test_small_betas(cuda_lib, N, P, gate, segments):
    """Every beta near sigmoid(gate), no state to begin with: y and the state are as
    small as the betas, and as exact as otherwise."""
    inp = make(N, P, L=330, B=1)
    inp["b_raw"] = (gate + 0.5 * inp["b_raw"].float()).bfloat16()
    y, h = run(inp, h0=False, segments=segments)
    y_ref, h_ref = ref(inp, h0=False)
    size = np.exp(gate)
    close(y / size, y_ref / size, 2.6e-3, "y", 1.3e-2)
    close(h / size, h_ref / size, 1e-5, "state")


@pytest.mark.parametrize("segments", [1, 3])
def test_betas_of_every_size(cuda_lib, segments):
    """Chunks of large and of small betas in turn, one with none at all, each head after its own pattern."""
    inp = make(L=450, B=2)
    gates = torch.tensor([[0., -14., -4., -90., 3., -9., 1., -25.], [-14., 0., -30., 2., -6., -6., 5., 0.],
                          [-20., -16., -12., -8., -4., 0., 0., 0.], [0., -4., -8., -12., -16., -20., -24., -28.]])
    inp["b_raw"] = (inp["b_raw"].float() + gates.repeat_interleave(64, 1)[:, :450].T).bfloat16()
    inp["b_raw"][:, 64:128, 3] = -float("inf")
    want = {n: t.clone() for n, t in inp.items()}
    want["b_raw"][:, 64:128, 3] = -1e4
    for h0 in (False, True):
        y, h = run(inp, h0=h0, segments=segments)
        y_ref, h_ref = ref(want, h0=h0)
        for hd in range(4):
            close(y[:, :, hd], y_ref[:, :, hd], 2.6e-3, f"y of head {hd}", 1.3e-2)
            close(h[:, hd], h_ref[:, hd], 1e-5, f"state of head {hd}")


# ------------------------------------------------------------ long memories token by token
SLOW = [(-3.0, None), (-6.0, -4.0), (-8.0, -4.0), (-8.0, None), (-10.0, -4.0), (-14.0, -9.0)]


def slow(db, b, L, io="f32", const=True):
    """Tokens whose decays are all alike and keep some e^-db of them, and which replace little."""
    inp = make(64, 128, G=1, H=2, io=io, L=L, B=1)
    inp["dt_bias"][:] = torch.tensor([db, db - 1])
    inp["A_log"][:] = 0.0
    if const:
        inp["dt_raw"][:] = 0.3
    if b is not None:
        inp["b_raw"][:] = b
    return inp


def slow_tol(db, n):
    """An element of the state is rounded three times a token, to either side: sqrt(3 n)
    2^-25 / sqrt(3), 2e-6 of n = 4096, asserted at 1e-5.  But where a token takes off few
    steps of an element, S - (1 - a) S with (1 - a) < 2^-17, or 2^7 steps of 2^-24 at most,
    the difference is rounded the same way at token after token until the element has
    changed by a good part of itself, which it does not: at most half a step, 2^-24 of the
    element, n times.  That is the float32 state's own limit, whatever a is known to."""
    return 1e-5 if np.exp(db - 1) >= 2 ** -17 else n * 2 ** -24


@pytest.mark.parametrize("const", [True, False])
@pytest.mark.parametrize("db, b", SLOW)
def test_long_memory_token_by_token(cuda_lib, db, b, const):
    inp, tol = slow(db, b, 4096, const=const), slow_tol(db, 4096)
    y, h = run(inp)
    y_ref, h_ref = ref(inp)
    close(y, y_ref, tol, "y")
    close(h, h_ref, tol, "state")


@pytest.mark.parametrize("db, b", SLOW)
def test_long_memory_of_steps(cuda_lib, db, b):
    from selective_state_space_52_b200 import axon_ssm
    inp = slow(db, b, 3000)
    d, params = dev(inp)
    state = d["h0"].clone()
    seq = [d[n].unbind(1) for n in SEQ]
    ys = [axon_ssm.delta_step(*t, params, state) for t in zip(*seq)]
    y_ref, h_ref = ref(inp)
    close(torch.stack(ys, 1).cpu().numpy(), y_ref, slow_tol(db, 3000), "y")
    close(state.cpu().numpy(), h_ref, slow_tol(db, 3000), "state")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_every_rate_of_decay(cuda_lib, io):
    """Decays of one token from 1 to 0 past the middle, where the state's form of it changes; no writes beside them."""
    L = 40
    inp = make(G=1, H=4, io=io, L=L, B=1)
    inp["A_log"][:] = 0.0
    inp["dt_bias"][:] = torch.tensor([-20.0, -0.001, 0.001, 4.0])
    inp["dt_raw"] = torch.linspace(-1, 1, L)[None, :, None].expand(1, L, 4).to(inp["dt_raw"].dtype).contiguous()
    inp["v"][:] = 0
    inp["b_raw"][:] = -100.0
    want, _ = ref(inp)
    y, h = run(inp)
    for t in range(12):
        close(y[:, t], want[:, t], tols(io)[0], f"y of token {t}", 4e-4 if io == "f32" else 1.3e-2)
        for hd in range(4):
            r = want[0, t, hd]
            assert np.linalg.norm(y[0, t, hd] - r) <= (3e-5 if io == "f32" else 2.6e-3) * np.linalg.norm(r) + 1e-36, (t, hd)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_bindings_of_the_c_entries(cuda_lib, io):
    """The binding's functions of the C names, called with every argument, as the convenience calls give them."""
    from selective_state_space_52_b200 import axon_ssm
    inp = make(64, 128, 2, 4, io, L=130, B=2)
    d, params = dev(inp)
    code = axon_ssm.AXON_F32 if io == "f32" else axon_ssm.AXON_BF16
    gates = (d["dt_raw"], d["b_raw"], d["dt_bias"], d["A_log"])
    qkv = (d["q"], 128, d["k"], 128, d["v"], 512)
    lengths = torch.tensor([130, 77], dtype=torch.int32, device="cuda")
    n = axon_ssm.axon_delta_workspace_bytes(2, 130, 4, 2, 128, 64, code, 2 if io == "bf16" else 0)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    y, h = torch.zeros_like(d["v"]), torch.empty_like(d["h0"])
    seg = 2 if io == "bf16" else 0
    assert axon_ssm.axon_delta_scan_fwd(2, 130, 4, 2, 128, 64, code, *qkv, *gates, lengths, d["h0"], 0.3, 1, y, h, seg, ws, n) == 0
    want = axon_ssm.delta_scan(*(d[m] for m in SEQ), params, d["h0"], lengths=lengths, scale=0.3, segments=seg,
                               out=(torch.zeros_like(y), torch.empty_like(h)))
    assert torch.equal(y, want[0]) and torch.equal(h, want[1])
    one = [d[m][:, 5].contiguous() for m in SEQ]
    y1, s1, s2 = torch.empty_like(one[2]), d["h0"].clone(), d["h0"].clone()
    axon_ssm.axon_delta_step(2, 4, 2, 128, 64, code, one[0], 128, one[1], 128, one[2], 512, one[3], one[4], d["dt_bias"],
                             d["A_log"], 0.3, 0, s1, y1)
    y2 = axon_ssm.delta_step(*one, params, s2, scale=0.3, qk_norm=False)
    assert torch.equal(y1, y2) and torch.equal(s1, s2)
    x, z, w, b = d["v"].flatten(2), d["v"].flatten(2).flip(1).contiguous(), torch.rand(512, device="cuda"), torch.rand(512, device="cuda")
    o = torch.empty_like(x)
    axon_ssm.axon_gated_norm_fwd(260, 512, 128, code, 1, 2, 1, x, 512, z, 512, w, b, 1, 1e-5, o, 512)
    assert torch.equal(o, axon_ssm.gated_norm(x, w, z, bias=b, group=128, kind="group", gate="before", eps=1e-5))
