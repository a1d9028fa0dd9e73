"""The gated delta rule and the grouped gated norm without a GPU: the fp64
oracle against forms that share nothing with its loop, and the C ABI's and the
binding's refusals (fake, never dereferenced pointers: every call fails
argument validation, so nothing is launched)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle

FAKE = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from selective_state_space_52_b200 import build
    build.build()
    from selective_state_space_52_b200 import axon_ssm
    return axon_ssm._lib


# ------------------------------------------------------------ oracle pins
def rand_delta(rng, B=2, L=23, G=2, H=4, P=5, N=6):
    return dict(q=rng.standard_normal((B, L, G, N)), k=rng.standard_normal((B, L, G, N)),
                v=rng.standard_normal((B, L, H, P)), dt_raw=rng.standard_normal((B, L, H)),
                b_raw=rng.standard_normal((B, L, H)), dt_bias=rng.standard_normal(H) - 3,
                A_log=rng.standard_normal(H), h0=rng.standard_normal((B, H, P, N)))


def test_delta_matches_matrix_products():
    """S_t as explicit products with a (I - beta k^ k^^T): numpy matrices."""
    rng = np.random.default_rng(1)
    d = rand_delta(rng)
    y, h = oracle.delta_scan(**d)
    B, L, H, P = d["v"].shape
    N = d["k"].shape[-1]
    for b in range(B):
        for hd in range(H):
            S = d["h0"][b, hd]
            for t in range(L):
                k, q = d["k"][b, t, hd // 2], d["q"][b, t, hd // 2]
                k, q = (u / np.linalg.norm(np.append(u, 1e-3)) for u in (k, q))
                a = np.exp(-np.exp(d["A_log"][hd]) * np.log1p(np.exp(d["dt_raw"][b, t, hd] + d["dt_bias"][hd])))
                beta = 0.5 * (1 + np.tanh(d["b_raw"][b, t, hd] / 2))
                S = a * S @ (np.eye(N) - beta * np.outer(k, k)) + beta * np.outer(d["v"][b, t, hd], k)
                np.testing.assert_allclose(y[b, t, hd], S @ q / np.sqrt(N), rtol=1e-11, atol=1e-12)
            np.testing.assert_allclose(h[b, hd], S, rtol=1e-11, atol=1e-12)


def test_delta_replaces_what_a_key_held():
    """beta = 1, no decay, unit keys: reading a key returns the last value written to it."""
    N = P = 4
    k = np.eye(N)[[0, 1, 0, 2, 1]][None, :, None]
    v = np.random.default_rng(2).standard_normal((1, 5, 1, P))
    y, h = oracle.delta_scan(k, k, v, np.full((1, 5, 1), -800.0), np.full((1, 5, 1), 800.0), np.zeros(1), np.zeros(1),
                             norm=False, scale=1.0)
    np.testing.assert_allclose(y, v, atol=1e-14)
    np.testing.assert_allclose(h[0, 0].T, np.stack([v[0, 2, 0], v[0, 4, 0], v[0, 3, 0], np.zeros(P)]), atol=1e-14)


def test_delta_split_sequence_and_lengths():
    d = rand_delta(np.random.default_rng(3), L=17)
    y, h = oracle.delta_scan(**d)
    cut = {n: t[:, :6] if t.ndim > 2 and n != "h0" else t for n, t in d.items()}
    y1, h1 = oracle.delta_scan(**cut)
    rest = {n: t[:, 6:] if t.ndim > 2 and n != "h0" else t for n, t in d.items()}
    y2, h2 = oracle.delta_scan(**{**rest, "h0": h1})
    np.testing.assert_array_equal(np.concatenate([y1, y2], 1), y)
    np.testing.assert_array_equal(h2, h)
    y3, h3 = oracle.delta_scan(**d, lengths=np.array([6, 0]))
    np.testing.assert_array_equal(y3[0, :6], y1[0])
    np.testing.assert_array_equal(h3, np.stack([h1[0], d["h0"][1]]))
    assert not y3[0, 6:].any() and not y3[1].any()


@pytest.mark.parametrize("kind", ["rms", "group"])
@pytest.mark.parametrize("gate", [None, "after", "before"])
def test_gated_norm_matches_torch(kind, gate):
    g = torch.Generator().manual_seed(4)
    x, z = (torch.randn(5, 24, generator=g, dtype=torch.float64) for _ in range(2))
    w, b = (torch.randn(24, generator=g, dtype=torch.float64) for _ in range(2))
    silu = torch.nn.functional.silu
    t = x * silu(z) if gate == "before" else x
    if kind == "group":
        o = torch.nn.functional.group_norm(t, 3, w, b, 1e-5)
    else:
        o = torch.nn.functional.rms_norm(t.view(5, 3, 8), (8,), eps=1e-5).view(5, 24) * w + b
    o = o * silu(z) if gate == "after" else silu(o) if gate is None else o
    got = oracle.gated_norm(x, 8, kind, gate, True, z, w, b, 1e-5)
    np.testing.assert_allclose(got, o.numpy(), rtol=1e-12, atol=1e-13)


# ------------------------------------------------------------ refusals of the C ABI
def scan(lib, **over):
    a = dict(B=1, L=64, H=4, G=2, P=64, N=128, io=1, q=FAKE, ldq=256, k=FAKE + (1 << 24), ldk=256, v=FAKE + (2 << 24),
             ldv=256, dt_raw=FAKE + (3 << 24), b_raw=FAKE + (4 << 24), dt_bias=FAKE + (5 << 24),
             A_log=FAKE + (6 << 24), lengths=None, h0=None, scale=0.1, norm=1, y=FAKE + (7 << 24),
             h_out=FAKE + (8 << 24), segments=1, workspace=FAKE + (9 << 24), workspace_bytes=1 << 24, stream=None)
    a.update(over)
    return lib.axon_delta_scan_fwd(*a.values())


@pytest.mark.parametrize("over, status", [
    (dict(B=-1), 1), (dict(L=-1), 1), (dict(H=-1), 1), (dict(segments=-1), 1),
    (dict(workspace_bytes=1000), 4), (dict(workspace=None), 1), (dict(workspace=FAKE + (9 << 24) + 8), 3),
    (dict(workspace=FAKE + (7 << 24) + 4096), 1),
    (dict(H=5), 2), (dict(G=0), 2), (dict(P=32), 2), (dict(N=96), 2), (dict(io=2), 2), (dict(B=70000), 2),
    (dict(L=1 << 30), 2),
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(dt_raw=None), 1), (dict(b_raw=None), 1),
    (dict(dt_bias=None), 1), (dict(A_log=None), 1), (dict(y=None), 1), (dict(h_out=None), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(ldq=248), 1), (dict(ldk=128), 1), (dict(ldv=255), 1),
    (dict(ldq=260), 3), (dict(ldv=257), 3), (dict(q=FAKE + 8), 3), (dict(y=FAKE + (7 << 24) + 2), 3),
    (dict(h0=FAKE + (10 << 24) + 4), 3), (dict(lengths=FAKE + (10 << 24) + 2), 3), (dict(io=0, ldq=258), 3),
    (dict(y=FAKE), 1), (dict(y=FAKE + (2 << 24)), 1), (dict(h_out=FAKE + (1 << 24)), 1),
    (dict(y=FAKE + (8 << 24)), 1), (dict(h0=FAKE + (8 << 24) + 64), 1), (dict(lengths=FAKE + (7 << 24)), 1),
    (dict(h_out=FAKE + (6 << 24)), 1),
])
def test_delta_scan_rejects(lib, over, status):
    assert scan(lib, **over) == status


def test_delta_scan_rejects_strided_overlap(lib):
    # 64 tokens 4096 elements apart reach 516096 bytes in: y in a gap between two tokens still lies inside
    assert scan(lib, ldv=4096, y=FAKE + (2 << 24) + 4096 * 2 * 62 + 1024) == 1


def test_delta_workspace_query(lib):
    q = lib.axon_delta_workspace_bytes
    chunk = lambda G, H, N: G * 128 * N * 2 + H * 25600             # noqa: E731
    # whole sequences: the flag's 256 bytes and every chunk's tiles
    assert q(1, 640, 4, 2, 128, 128, 1, 1) == 256 + 10 * chunk(2, 4, 128)
    assert q(3, 65, 5, 5, 64, 64, 1, 1) == 256 + 6 * chunk(5, 5, 64)
    # three segments: two end states, one transition with its row scales, h0 again
    state = 4 * 64 * 128 * 4
    assert q(1, 640, 4, 2, 64, 128, 1, 3) == 256 + 10 * chunk(2, 4, 128) + 2 * state + 4 * 4 * 128 * 128 + 4 * 128 * 4 + state
    assert q(1, 640, 4, 2, 128, 128, 0, 0) == 0                     # float32: token by token
    assert q(1, 8, 4, 2, 128, 128, 1, 0) == 0                       # so are a few tokens, if nothing else is asked for
    assert q(1, 8, 4, 2, 128, 128, 1, 1) == 256 + chunk(2, 4, 128)
    assert q(1, 1000, 4, 2, 128, 128, 1, 0) > 0
    for bad in ((-1, 64, 4, 2, 128, 128, 1, 0), (1, 64, 5, 2, 128, 128, 1, 0), (1, 64, 4, 2, 96, 128, 1, 0),
                (1, 64, 4, 2, 128, 128, 1, -1)):
        assert q(*bad) == 0


def test_delta_noop_sizes(lib):
    assert scan(lib, B=0) == 0
    assert scan(lib, H=0) == 0


def step(lib, **over):
    a = dict(B=2, H=4, G=2, P=64, N=128, io=1, q=FAKE, ldq=256, k=FAKE + (1 << 24), ldk=256, v=FAKE + (2 << 24),
             ldv=256, dt_raw=FAKE + (3 << 24), b_raw=FAKE + (4 << 24), dt_bias=FAKE + (5 << 24),
             A_log=FAKE + (6 << 24), scale=0.1, norm=1, state=FAKE + (7 << 24), y=FAKE + (8 << 24), stream=None)
    a.update(over)
    return lib.axon_delta_step(*a.values())


@pytest.mark.parametrize("over, status", [
    (dict(B=-1), 1), (dict(H=6, G=4), 2), (dict(P=48), 2), (dict(N=256), 2), (dict(io=7), 2), (dict(B=1 << 20), 2),
    (dict(q=None), 1), (dict(state=None), 1), (dict(y=None), 1), (dict(ldk=16), 1), (dict(ldk=257), 3),
    (dict(state=FAKE + (7 << 24) + 8), 3), (dict(y=FAKE), 1), (dict(state=FAKE + (2 << 24)), 1),
    (dict(y=FAKE + (7 << 24) + 256), 1), (dict(scale=float("nan")), 1),
])
def test_delta_step_rejects(lib, over, status):
    assert step(lib, **over) == status
    assert step(lib, B=0) == 0


def norm(lib, **over):
    a = dict(rows=8, C=256, D=64, io=1, kind=0, gate=1, act=1, x=FAKE, ldx=256, z=FAKE + (1 << 24), ldz=256,
             w=FAKE + (2 << 24), b=None, per_channel=0, eps=1e-6, y=FAKE + (3 << 24), ldy=256, stream=None)
    a.update(over)
    return lib.axon_gated_norm_fwd(*a.values())


@pytest.mark.parametrize("over, status", [
    (dict(rows=-1), 1), (dict(D=0), 1), (dict(D=-64), 1), (dict(D=96), 1), (dict(C=-256), 1), (dict(io=2), 2),
    (dict(kind=2), 2), (dict(gate=3), 2), (dict(C=16384, D=16384, ldx=16384, ldy=16384, ldz=16384), 2),
    (dict(rows=1 << 30, D=8), 2), (dict(rows=(1 << 31) - 1, D=256), 2), (dict(rows=(1 << 29) - 1), 2), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(x=None), 1), (dict(z=None), 1), (dict(y=None), 1), (dict(ldx=128), 1), (dict(ldz=248), 1), (dict(ldy=0), 1),
    (dict(C=260, D=4, ldx=264, ldz=264, ldy=264), 3), (dict(ldx=260), 3), (dict(x=FAKE + 2), 3), (dict(w=FAKE + (2 << 24) + 4), 3),
    (dict(y=FAKE + 512), 1), (dict(ldx=512, ldy=512, y=FAKE + 256), 1), (dict(ldx=512, ldy=512, y=FAKE + 768 + 4096), 1), (dict(y=FAKE, ldy=512), 1), (dict(y=FAKE + (1 << 24) + 1024), 1), (dict(y=FAKE + (2 << 24)), 1),
])
def test_gated_norm_rejects(lib, over, status):
    assert norm(lib, **over) == status


def test_gated_norm_noop_sizes(lib):
    assert norm(lib, rows=0) == 0
    assert norm(lib, C=0) == 0


# ------------------------------------------------------------ refusals of the binding
def test_binding_refuses_cpu_tensors(lib):
    from selective_state_space_52_b200 import axon_ssm
    t = torch.zeros(1, 4, 2, 64)
    r = torch.zeros(1, 4, 2)
    params = {"dt_bias": torch.zeros(2), "A_log": torch.zeros(2)}
    with pytest.raises(ValueError, match="CUDA device"):
        axon_ssm.delta_scan(t, t, t, r, r, params)
    with pytest.raises(ValueError, match="CUDA device"):
        axon_ssm.delta_step(t[:, 0], t[:, 0], t[:, 0], r[:, 0], r[:, 0], params, torch.zeros(1, 2, 64, 64))
    with pytest.raises(ValueError, match="CUDA device"):
        axon_ssm.gated_norm(torch.zeros(4, 64))


def test_binding_token_strides(lib):
    from selective_state_space_52_b200.axon_ssm import _row_stride, _token_stride
    row = torch.zeros(2, 5, 10 * 64)
    q, k, v = row[..., :128].view(2, 5, 2, 64), row[..., 128:256].view(2, 5, 2, 64), row[..., 256:].view(2, 5, 6, 64)
    assert [_token_stride("f", "t", t) for t in (q, k, v)] == [640] * 3
    assert _token_stride("f", "t", v[:, :1]) == 3200                # one token a row: the rows' own stride
    assert _token_stride("f", "t", v[:1, :1]) == 6 * 64             # one token in all: any stride will do
    assert _token_stride("f", "t", q[:, 0]) == 3200
    for bad in (q[:, ::1, :, ::2], row.view(2, 5, 10, 64)[:, :, ::2], row.view(2, 5, 10, 64)[:, :4], q.transpose(0, 1)):
        with pytest.raises(ValueError):
            _token_stride("f", "t", bad)
    assert _row_stride("f", "t", row[..., :128], 10, 128) == 640
    assert _row_stride("f", "t", row[0, :, 128:], 5, 512) == 640
    with pytest.raises(ValueError):
        _row_stride("f", "t", row[:, :4, :128], 8, 128)
    with pytest.raises(ValueError):
        _row_stride("f", "t", row[..., ::2], 10, 320)


@pytest.fixture
def recorded(lib, monkeypatch):
    """The binding on CPU tensors with a recorder in place of the library: what would be launched, launched nowhere."""
    from selective_state_space_52_b200 import axon_ssm
    calls = []

    class Recorder:
        def __getattr__(self, name):
            def call(*args):
                calls.append((name, args))
                return 0
            return call

    monkeypatch.setattr(axon_ssm, "_lib", Recorder())
    monkeypatch.setattr(axon_ssm, "_same_device", lambda what, dev, **tensors: None)
    monkeypatch.setattr(axon_ssm, "_current_device", lambda: -1)
    monkeypatch.setattr(axon_ssm, "_stream_on", lambda stream, index: None)
    return axon_ssm, calls


def delta_tensors(*lead, G=2, H=4, P=64, N=64):
    def t(*shape):
        return torch.zeros(*lead, *shape, dtype=torch.bfloat16)
    params = {"dt_bias": torch.zeros(H), "A_log": torch.zeros(H)}
    return t(G, N), t(G, N), t(H, P), t(H), t(H), params


@pytest.mark.parametrize("lead", [(), (4,), (2, 3, 5), (1, 2, 3, 5)])
def test_delta_scan_refuses_other_ranks(recorded, lead):
    """A step's tensors or a prompt without its batch dimension would pass heads for tokens."""
    axon_ssm, calls = recorded
    with pytest.raises(ValueError, match="dimensions"):
        axon_ssm.delta_scan(*delta_tensors(*lead))
    assert not calls


@pytest.mark.parametrize("lead", [(), (2, 1), (2, 3), (2, 3, 5)])
def test_delta_step_refuses_other_ranks(recorded, lead):
    axon_ssm, calls = recorded
    with pytest.raises(ValueError, match="dimensions"):
        axon_ssm.delta_step(*delta_tensors(*lead), torch.zeros(2, 4, 64, 64))
    assert not calls


@pytest.mark.parametrize("which", [0, 1, 2, 3, 4])
def test_delta_refuses_one_tensor_of_another_rank(recorded, which):
    axon_ssm, calls = recorded
    args = list(delta_tensors(2, 8))
    for bad in (args[which][0], args[which][None], args[which].flatten()[0]):
        with pytest.raises(ValueError):
            axon_ssm.delta_scan(*args[:which], bad, *args[which + 1:])
    assert not calls


def test_delta_right_ranks_reach_the_library(recorded):
    axon_ssm, calls = recorded
    axon_ssm.delta_scan(*delta_tensors(2, 8), check=False)
    axon_ssm.delta_step(*delta_tensors(3), torch.zeros(3, 4, 64, 64))
    scan_args, step_args = (a for n, a in calls if n != "axon_delta_workspace_bytes")
    assert scan_args[:6] == (2, 8, 4, 2, 64, 64) and step_args[:5] == (3, 4, 2, 64, 64)


# ------------------------------------------------------------ counts and strides that the C ABI's ints cannot hold
@pytest.mark.parametrize("shape, group", [(((1 << 32) + 5, 8), None), ((1 << 31, 8), None), ((1 << 16, 1 << 15, 16), 8),
                                          ((1, (1 << 32) + 64), None), ((1, (1 << 32) + 64), 64), ((3, 128), (1 << 32) + 64)])
def test_gated_norm_refuses_counts_past_31_bits(recorded, shape, group):
    """Only the low 32 bits would reach the library: 2^32 + 5 rows as 5."""
    axon_ssm, calls = recorded
    x = torch.empty(shape, dtype=torch.bfloat16, device="meta")
    with pytest.raises(axon_ssm.AxonError) as e:
        axon_ssm.gated_norm(x, group=group, out=x)
    assert e.value.status == 2 and not calls


def far_apart(stride, *tail):
    """Two rows (or one token of two batch rows) `stride` elements apart; no memory behind them."""
    return torch.empty(2 * stride, dtype=torch.bfloat16, device="meta").as_strided((2, *tail), (stride, *torch.empty(tail, device="meta").stride()))


@pytest.mark.parametrize("stride", [1 << 31, (1 << 32) + 128, (1 << 32) + 4096])
def test_strides_past_31_bits_are_refused(recorded, stride):
    axon_ssm, calls = recorded
    wide, x = far_apart(stride, 128), torch.empty(2, 128, dtype=torch.bfloat16, device="meta")
    for kw in (dict(x=wide, out=x), dict(x=x, z=wide, out=x), dict(x=x, out=wide)):
        with pytest.raises(ValueError, match="stride"):
            axon_ssm.gated_norm(group=64, **kw)
    q, k, v, dt_raw, b_raw, params = (t if isinstance(t, dict) else t.to("meta") for t in delta_tensors(2))
    state = torch.empty(2, 4, 64, 64, device="meta")
    for n, t in enumerate((far_apart(stride, 2, 64), far_apart(stride, 2, 64), far_apart(stride, 4, 64))):
        args = [q, k, v]
        args[n] = t
        with pytest.raises(ValueError, match="stride"):
            axon_ssm.delta_step(*args, dt_raw, b_raw, params, state)
        with pytest.raises(ValueError, match="stride"):
            axon_ssm.delta_scan(*(u[:, None] for u in (*args, dt_raw, b_raw)), params, check=False)
    assert not calls


def test_the_largest_stride_passes(lib):
    from selective_state_space_52_b200.axon_ssm import _row_stride, _token_stride
    last = (1 << 31) - 8
    assert _row_stride("f", "t", far_apart(last, 128), 2, 128) == last
    assert _token_stride("f", "t", far_apart(last, 2, 64)) == last


# ------------------------------------------------------------ alignment: what the kernels' loads need, no more
GATES = dict(dt_raw=3, b_raw=4)
PARAMS = dict(dt_bias=5, A_log=6)


@pytest.mark.parametrize("call", [scan, step])
@pytest.mark.parametrize("io", [0, 1])
@pytest.mark.parametrize("name", [*GATES, *PARAMS])
def test_delta_rates_need_their_own_alignment(lib, call, io, name):
    """A value's own alignment passes (the call then fails for y over q), less does not."""
    at = FAKE + ({**GATES, **PARAMS}[name] << 24)
    size = 2 if io == 1 and name in GATES else 4
    assert call(lib, io=io, **{name: at + size}, y=FAKE) == 1
    assert call(lib, io=io, **{name: at + size // 2}, y=FAKE) == 3


@pytest.mark.parametrize("B, L, H, P, N, chunks", [
    # measured on the device, us token by token and in chunks: wherever one takes a fifth more, the other is chosen
    (1, 96, 8, 128, 128, False), (1, 160, 1, 128, 128, True), (1, 160, 8, 64, 128, True), (1, 112, 1, 64, 64, True),
    (1, 80, 8, 64, 64, False), (1, 128, 8, 64, 64, True), (8, 32, 32, 128, 64, False), (8, 48, 32, 64, 64, False),
    (8, 48, 16, 128, 128, True), (32, 24, 32, 128, 128, False), (32, 48, 32, 128, 128, True), (32, 48, 32, 64, 64, False),
    (32, 128, 32, 64, 64, True),
])
def test_delta_path_is_the_faster_one(lib, B, L, H, P, N, chunks):
    assert (lib.axon_delta_workspace_bytes(B, L, H, 1, P, N, 1, 0) > 0) == chunks


def test_delta_wait_probe_rejects_bad_arguments(lib):
    f = lib.axon_delta_wait_probe
    for status, limit, want in ((None, 64, 1), (FAKE, 0, 1), (FAKE, -5, 1), (FAKE, (1 << 16) + 1, 1), (FAKE + 2, 64, 1)):
        assert f(status, limit, None) == want
