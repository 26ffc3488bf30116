"""Decayed linear attention (linear_prefill, linear_decode) against its
definition in 64 bits, element by element, within bounds derived in
tests/_linear_ref.py.

Outputs are pre-filled with NaN, so an element that a kernel does not write
fails. The lengths go around the kernels' block sizes (32, 64, 128 tokens) and
the decays through the values where exponents go wrong: none, strong ones,
resets (-infinity), positive ones, one fixed for each head.
"""
import ctypes

import numpy as np
import pytest
import torch

from tests import _linear_ref as ref

gdn = pytest.importorskip("gated_deltanet_linear_21_b200")

DEV = "cuda"
P = 0x10000  # a 16-byte aligned fake device address (never dereferenced)
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def decays(kind, T, Hv, gen):
    if kind == "fixed":
        return torch.log1p(-torch.exp2(-2.0 - 8 * torch.rand(Hv, generator=gen)))
    g = torch.nn.functional.logsigmoid(torch.randn(T, Hv, generator=gen) + 3)
    if kind == "none":
        g[:] = 0.0
    elif kind == "strong":
        g = torch.randn(T, Hv, generator=gen) * 0.5 - 5
    elif kind == "reset":
        g[torch.rand(T, Hv, generator=gen) < 0.05] = -float("inf")
    elif kind == "far":
        g[torch.rand(T, Hv, generator=gen) < 0.05] = -1e4
    elif kind == "positive":
        g[torch.rand(T, Hv, generator=gen) < 0.1] = 0.05
    return g


def draw(lengths, Hqk, Hv, dk, dv, dtype, kind="token", init=True, seed=0, front=0, behind=0):
    gen = torch.Generator().manual_seed(7000 + seed + sum(lengths))
    T = front + sum(lengths) + behind
    x = dict(q=torch.randn(T, Hqk, dk, generator=gen).to(dtype), k=torch.randn(T, Hqk, dk, generator=gen).to(dtype),
             v=torch.randn(T, Hv, dv, generator=gen).to(dtype), g=decays(kind, T, Hv, gen).float(),
             state_in=torch.randn(len(lengths), Hv, dv, dk, generator=gen) if init else None,
             cu=torch.tensor([front] + lengths, dtype=torch.int64).cumsum(0).to(torch.int32))
    return x


def on_gpu(x):
    return {n: t.to(DEV) if t is not None else None for n, t in x.items()}


def prefill(x, **kw):
    d = on_gpu(x)
    T, Hv, dv = x["v"].shape
    N, dk = x["cu"].numel() - 1, x["q"].shape[2]
    o = torch.full((T, Hv, dv), float("nan"), dtype=x["q"].dtype, device=DEV)
    s = torch.full((N, Hv, dv, dk), float("nan"), device=DEV)
    gdn.linear_prefill(d["q"], d["k"], d["v"], d["g"], d["state_in"], d["cu"], o=o, state_out=s, **kw)
    torch.cuda.synchronize()
    gdn.device_error()
    return o, s


def check(x, o, s, scale=None):
    ro, rs, mo, ms = ref.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["state_in"], x["cu"], scale)
    T, a, b = ref.steps(x["cu"]), int(x["cu"][0]), int(x["cu"][-1])
    ref.check_o(o[a:b], ro[a:b], mo[a:b], T, x["q"].shape[2])
    ref.check_state(s, rs, ms, T)


# ----------------------------------------------------------------- prefill ---

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("lengths", [[1], [2], [31], [32], [33], [64], [127], [128], [129], [255], [257], [700],
                                     [0, 5, 0, 0, 130, 1], [128, 128], [300, 64, 0, 1, 257]], ids=str)
def test_prefill_lengths(dtype, lengths):
    x = draw(lengths, 2, 4, 128, 128, dtype)
    check(x, *prefill(x))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("dk,dv", [(16, 16), (32, 64), (64, 32), (128, 16), (16, 128), (64, 64), (128, 64)])
def test_prefill_head_sizes(dtype, dk, dv):
    x = draw([133, 40], 2, 2, dk, dv, dtype, seed=1)
    check(x, *prefill(x))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("kind", ["none", "strong", "reset", "far", "positive", "fixed"])
def test_prefill_decays(dtype, kind):
    x = draw([290, 3, 128], 1, 3, 128, 128, dtype, kind, seed=2)
    check(x, *prefill(x))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prefill_without_a_state_and_with_a_scale(dtype):
    x = draw([200, 17], 2, 8, 128, 128, dtype, init=False, seed=3)
    check(x, *prefill(x, scale=0.5), scale=0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_prefill_over_many_blocks(dtype):
    """Sequences long enough that the work of one head is split over time."""
    x = draw([2500, 1], 1, 2, 128, 128, dtype, "fixed", seed=4)
    check(x, *prefill(x))
    x = draw([1900, 700], 1, 1, 128, 128, dtype, seed=5)
    check(x, *prefill(x))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_rows_outside_the_sequences_stay_and_do_not_matter(dtype):
    x = draw([130, 0, 70], 2, 2, 128, 128, dtype, front=5, behind=150, seed=6)
    a, b = int(x["cu"][0]), int(x["cu"][-1])
    for n in ("q", "k", "v", "g"):
        x[n][:a] = float("nan")
        x[n][b:] = float("nan")
    d = on_gpu(x)
    o = torch.full(x["v"].shape, 7.0, dtype=dtype, device=DEV)
    _, s = gdn.linear_prefill(d["q"], d["k"], d["v"], d["g"], d["state_in"], d["cu"], o=o)
    gdn.device_error()
    assert (o[:a] == 7).all() and (o[b:] == 7).all()
    check(x, o, s)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_sequence_of_infinities_leaves_its_neighbours_alone(dtype, bad):
    x = draw([70, 200, 131], 1, 2, 128, 128, dtype, seed=7)
    x["k"][70:270] = bad
    x["v"][70:270] = bad
    x["state_in"][1] = bad
    o, s = prefill(x)
    keep = [0, 2]
    y = {n: t for n, t in x.items()}
    for n in ("k", "v"):
        y[n] = x[n].clone()
        y[n][70:270] = 0
    y["state_in"] = x["state_in"].clone()
    y["state_in"][1] = 0
    ro, rs, mo, ms = ref.linear_prefill(y["q"], y["k"], y["v"], y["g"], y["state_in"], y["cu"])
    for i in keep:
        a, b = int(x["cu"][i]), int(x["cu"][i + 1])
        ref.check_o(o[a:b], ro[a:b], mo[a:b], 200, 128)
        ref.check_state(s[i], rs[i], ms[i], 200)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_state_out_may_be_state_in(dtype):
    x = draw([700, 0, 40], 1, 2, 128, 128, dtype, seed=8)
    o, s = prefill(x)
    d = on_gpu(x)
    o2, s2 = gdn.linear_prefill(d["q"], d["k"], d["v"], d["g"], d["state_in"], d["cu"], state_out=d["state_in"])
    gdn.device_error()
    assert s2 is d["state_in"] and torch.equal(o, o2) and torch.equal(s, s2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_large_values_keep_their_range(dtype):
    """Scores and states far outside f16's range, with outputs inside it."""
    x = draw([400], 1, 2, 128, 128, dtype, "none", init=False, seed=9)
    x["q"] = (x["q"].float() * 2.0 ** -7).to(dtype)
    x["k"] = (x["k"].float() * 64).to(dtype)
    x["v"] = (x["v"].float() * 64).to(dtype)
    o, s = prefill(x, scale=2.0 ** -6)
    assert torch.isfinite(o).all() and s.abs().max() > 65504
    check(x, o, s, scale=2.0 ** -6)


@pytest.mark.gpu
def test_a_broken_cu_seqlens_reads_and_writes_nothing_outside():
    x = draw([60, 60], 1, 2, 128, 128, BF16, seed=10)
    for cu in ([-5, 50, 4000], [90, 20, 120], [200, 300, 400]):
        x["cu"] = torch.tensor(cu, dtype=torch.int32)
        prefill(x)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cu", [[0, 4000, 0, 4000, 0, 4000], [0, 0, 4000, 10, 3990, -7, 5000]], ids=str)
def test_sequences_that_overlap_leave_what_is_behind_the_workspace(dtype, cu):
    """Offsets that go back make more segments than the workspace has room for."""
    x = draw([4000], 1, 2, 64, 64, dtype, init=False, seed=13)
    d, n = on_gpu(x), len(cu) - 1
    need = gdn.linear_prefill_workspace_bytes(n, 4000, 2, 64, 64, dtype)
    assert need > 0 and need % 16 == 0
    ws = torch.full((need + (64 << 20),), 171, dtype=torch.uint8, device=DEV)
    gdn.linear_prefill(d["q"], d["k"], d["v"], d["g"], None, torch.tensor(cu, dtype=torch.int32, device=DEV),
                       workspace=ws[:need])
    gdn.device_error()
    assert (ws[need:] == 171).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_repeated_captured_and_on_another_stream(dtype):
    x = draw([900, 130, 1], 2, 4, 128, 128, dtype, seed=11)
    o, s = prefill(x)
    for _ in range(3):
        o2, s2 = prefill(x)
        assert torch.equal(o, o2) and torch.equal(s, s2)
    d = on_gpu(x)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    o3, s3 = gdn.linear_prefill(d["q"], d["k"], d["v"], d["g"], d["state_in"], d["cu"], stream=other)
    other.synchronize()
    assert torch.equal(o, o3) and torch.equal(s, s3)
    # captured, with the inputs changed between replays
    y = on_gpu(draw([900, 130, 1], 2, 4, 128, 128, dtype, seed=12))
    o_y, s_y = gdn.linear_prefill(y["q"], y["k"], y["v"], y["g"], y["state_in"], y["cu"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        og, sg = gdn.linear_prefill(d["q"], d["k"], d["v"], d["g"], d["state_in"], d["cu"])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(og, o) and torch.equal(sg, s)
    for n in ("q", "k", "v", "g", "state_in"):
        d[n].copy_(y[n])
    graph.replay()
    torch.cuda.synchronize()
    gdn.device_error()
    assert torch.equal(og, o_y) and torch.equal(sg, s_y)


@pytest.mark.gpu
def test_two_calls_at_once():
    xs = [on_gpu(draw([1500, 20], 2, 8, 128, 128, BF16, seed=20 + i)) for i in range(2)]
    call = lambda x, st=None: gdn.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["state_in"], x["cu"], stream=st)  # noqa: E731
    want = [call(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        got = [call(x, st) for x, st in zip(xs, streams)]
        torch.cuda.synchronize()
        for (o, s), (ro, rs) in zip(got, want):
            assert torch.equal(o, ro) and torch.equal(s, rs)
    gdn.device_error()


# ------------------------------------------- prefill, split over time and heads ---

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("lengths,Hqk,Hv,dk,dv", [
    ([1300], 2, 20, 128, 128),                                  # more heads than one turn of the scan takes
    ([2600, 0, 1, 1500], 19, 38, 16, 32),
    ([0] * 3 + [1] * 40 + [1700] + [3] * 40 + [0] * 5 + [900], 2, 4, 64, 128),
    ([1500, 1100], 1, 1, 32, 16)], ids=["20 heads", "38 heads", "short around long", "one head"])
def test_prefill_split_over_time(dtype, lengths, Hqk, Hv, dk, dv):
    x = draw(lengths, Hqk, Hv, dk, dv, dtype, seed=50)
    check(x, *prefill(x))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_many_short_sequences(dtype):
    lengths = torch.randint(0, 4, (2500,), generator=torch.Generator().manual_seed(54)).tolist()
    x = draw(lengths, 1, 2, 16, 32, dtype, seed=54)
    check(x, *prefill(x))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("kind", ["strong", "reset", "far", "positive"])
def test_prefill_decays_across_segments(dtype, kind):
    x = draw([2300], 1, 2, 32, 64, dtype, kind, seed=51)
    if kind == "positive":      # 2300 tokens that grow would leave the range
        x["g"][300:] = 0.0
    check(x, *prefill(x))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_a_reset_and_bad_neighbours_across_segments(dtype):
    """A sequence of NaN that is split over time leaves the one behind it alone."""
    x = draw([1300, 1100], 1, 2, 64, 64, dtype, seed=52)
    want = {n: t.clone() for n, t in x.items()}
    x["k"][40:1290] = float("nan")
    x["state_in"][0] = float("inf")
    o, s = prefill(x)
    assert torch.isnan(o[1299]).all() and torch.isnan(s[0]).any()
    ro, rs, mo, ms = ref.linear_prefill(*(want[n] for n in ("q", "k", "v", "g", "state_in", "cu")))
    ref.check_o(o[1300:], ro[1300:], mo[1300:], 1100, 64)
    ref.check_state(s[1], rs[1], ms[1], 1100)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_two_graphs_that_share_a_workspace_replayed_in_turn(dtype):
    xs = [on_gpu(draw(n, 2, 4, 128, 128, dtype, seed=53)) for n in ([1900, 30], [700, 1400])]
    args = lambda x: (x["q"], x["k"], x["v"], x["g"], x["state_in"], x["cu"])  # noqa: E731
    want = [gdn.linear_prefill(*args(x)) for x in xs]
    need = max(gdn.linear_prefill_workspace_bytes(2, x["q"].shape[0], 4, 128, 128, dtype) for x in xs)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)     # its contents do not matter
    graphs, outs = [], []
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(gdn.linear_prefill(*args(x), workspace=ws))
        graphs.append(graph)
    for i in (0, 1, 1, 0, 1):
        outs[i][0].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i][0], want[i][0]) and torch.equal(outs[i][1], want[i][1])
    gdn.device_error()


@pytest.mark.gpu
def test_prefill_and_decode_beyond_32_bit_offsets():
    """v, o and the states have more than 2^31 elements; what lies behind them is checked."""
    T, tail, Hv, dk, dv = 131085, 300, 128, 16, 128
    small = draw([tail], 1, Hv, dk, dv, BF16, seed=54)
    d = on_gpu(small)
    q, k = (torch.zeros(T + tail, 1, dk, dtype=BF16, device=DEV) for _ in range(2))
    v, g = torch.zeros(T + tail, Hv, dv, dtype=BF16, device=DEV), torch.zeros(T + tail, Hv, device=DEV)
    for big, n in ((q, "q"), (k, "k"), (v, "v"), (g, "g")):
        big[T:] = d[n]
    state = torch.zeros(2, Hv, dv, dk, device=DEV)
    state[1] = d["state_in"][0]
    cu = torch.tensor([0, T, T + tail], dtype=torch.int32, device=DEV)
    assert v.numel() > 2 ** 31
    o, s = gdn.linear_prefill(q, k, v, g, state, cu)
    gdn.device_error()
    check(small, o[T:], s[1:])
    assert not o[T - 200:T].any() and not s[0].any()
    del v, o, q, k
    B, dk = 1030, 128
    y = on_gpu(draw([1], 1, Hv, dk, dv, BF16, seed=55))
    want_s = y["state_in"].clone()
    want_o = gdn.linear_decode(y["q"], y["k"], y["v"], y["g"], want_s)
    many = {n: y[n].expand(B, *y[n].shape[1:]).contiguous() for n in ("q", "k", "v", "g", "state_in")}
    assert many["state_in"].numel() > 2 ** 31
    o = gdn.linear_decode(many["q"], many["k"], many["v"], many["g"], many["state_in"])
    for b in (0, 1023, 1024, B - 1):
        assert torch.equal(o[b], want_o[0]) and torch.equal(many["state_in"][b], want_s[0])


# ------------------------------------------------------------------ decode ---

def decode_reference(x, state, scale=None):
    """One step: (o, S, mag_o, mag_S) through the prefill's definition, one token a sequence."""
    B = x["q"].shape[0]
    g = x["g"] if x["g"].dim() == 2 else x["g"].expand(B, -1)
    return ref.linear_prefill(x["q"], x["k"], x["v"], g, state, range(B + 1), scale)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("sdtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv,Hqk,Hv", [(16, 16, 1, 1), (32, 64, 2, 4), (64, 128, 1, 3), (128, 128, 2, 4), (128, 32, 2, 2)])
def test_decode(dtype, sdtype, dk, dv, Hqk, Hv):
    B = 5
    x = draw([1] * B, Hqk, Hv, dk, dv, dtype, "fixed" if Hv == 3 else "token", seed=30)
    state = x["state_in"].to(sdtype)
    d, sd = on_gpu(x), state.to(DEV)
    for _ in range(3):
        before = sd.cpu()
        o = torch.full((B, Hv, dv), float("nan"), dtype=dtype, device=DEV)
        gdn.linear_decode(d["q"], d["k"], d["v"], d["g"], sd, o=o)
        ro, rs, mo, ms = decode_reference(x, before)
        # o comes from the unrounded state: no operand of it is rounded to 16 bits
        u = torch.finfo(dtype).eps / 2
        ref._within(ref.f64(o), ro, u * np.abs(ro) + (dk + 8) * ref.F32 * mo, "o")
        ref.check_state(sd, rs, ms, 1)


@pytest.mark.gpu
def test_decode_follows_the_prefill_and_a_reset_forgets():
    x = draw([40, 40, 40], 2, 4, 128, 128, F32, seed=31)
    x["g"][59] = -float("inf")
    d = on_gpu(x)
    o, s = gdn.linear_prefill(d["q"], d["k"], d["v"], d["g"], d["state_in"], d["cu"])
    state = d["state_in"].clone()
    rows = torch.arange(3, device=DEV) * 40
    out = torch.empty_like(o)
    for t in range(40):
        i = rows + t
        out[i] = gdn.linear_decode(d["q"][i], d["k"][i], d["v"][i], d["g"][i], state)
    # the same recurrence in two orders of summation
    _, _, mo, ms = ref.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["state_in"], x["cu"])
    ref._within(ref.f64(out), ref.f64(o), 2 * (2 * 40 + 128 + 64) * ref.F32 * mo, "o")
    ref._within(ref.f64(state), ref.f64(s), 2 * (2 * 40 + 64) * ref.F32 * ms, "state")


@pytest.mark.gpu
def test_decode_captured_and_replayed():
    x = on_gpu(draw([1] * 9, 2, 4, 128, 128, BF16, seed=32))
    state, again = x["state_in"].clone(), x["state_in"].clone()
    gdn.linear_decode(x["q"], x["k"], x["v"], x["g"], again)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = gdn.linear_decode(x["q"], x["k"], x["v"], x["g"], state)
    for _ in range(2):
        want = gdn.linear_decode(x["q"], x["k"], x["v"], x["g"], again.copy_(state))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(state, again)


@pytest.mark.gpu
def test_empty_calls():
    z = lambda *s, dtype=BF16: torch.empty(*s, dtype=dtype, device=DEV)  # noqa: E731
    o = gdn.linear_decode(z(0, 2, 128), z(0, 2, 128), z(0, 4, 128), z(0, 4, dtype=F32), z(0, 4, 128, 128, dtype=F32))
    assert o.shape == (0, 4, 128)
    s0 = torch.randn(2, 4, 128, 128, device=DEV)
    cu = torch.zeros(3, dtype=torch.int32, device=DEV)
    o, s = gdn.linear_prefill(z(0, 2, 128), z(0, 2, 128), z(0, 4, 128), z(0, 4, dtype=F32), s0, cu)
    assert o.shape == (0, 4, 128) and torch.equal(s, s0)
    _, s = gdn.linear_prefill(z(0, 2, 128), z(0, 2, 128), z(0, 4, 128), z(0, 4, dtype=F32), None, cu)
    assert (s == 0).all()
    o, s = gdn.linear_prefill(z(0, 2, 128), z(0, 2, 128), z(0, 4, 128), z(0, 4, dtype=F32), None, cu[:1])
    assert s.shape == (0, 4, 128, 128)


# ---------------------------------------------------------------- refusals ---

@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_linear_21_b200 import build as gdn_build
    gdn_build.build()
    return gdn.lib()


def _c_prefill(lib, **kw):
    a = dict(q=P, k=P, v=P, g=P, g_stride=4, state_in=None, cu=P, n_seqs=1, total_T=64, Hqk=2, Hv=4, dk=128, dv=128,
             scale=0.0, dtype=gdn.GDN_BF16, o=P, state_out=P, ws=P, ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return lib.gdn_linear_prefill(*a.values())


def _c_decode(lib, name="gdn_linear_decode", **kw):
    a = dict(q=P, k=P, v=P, g=P, g_stride=4, state=P, B=4, Hqk=2, Hv=4, dk=128, dv=128, scale=0.0, dtype=gdn.GDN_BF16,
             o=P, stream=None)
    a.update(kw)
    return getattr(lib, name)(*a.values())


INV, UNS = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(g=None), INV), (dict(o=None), INV),
    (dict(cu=None), INV), (dict(state_out=None), INV), (dict(Hv=3), INV), (dict(Hqk=0), INV), (dict(n_seqs=-1), INV),
    (dict(total_T=-5), INV), (dict(total_T=1 << 31), INV), (dict(dk=96), UNS), (dict(dv=256), UNS), (dict(dtype=7), INV),
    (dict(q=P + 8), INV), (dict(state_in=P + 4), INV), (dict(g=P + 2), INV), (dict(g_stride=3), INV),
    (dict(g_stride=-4), INV), (dict(n_seqs=65536), UNS), (dict(Hqk=65536, Hv=65536, g_stride=0), UNS),
], ids=str)
def test_prefill_refuses(lib, kw, status):
    assert _c_prefill(lib, **kw) == status
    assert lib.gdn_last_error().decode().startswith("gdn_linear_prefill")


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_prefill_workspace_is_checked(lib, dtype):
    code = {BF16: gdn.GDN_BF16, F16: gdn.GDN_F16, F32: gdn.GDN_F32}[dtype]
    need = gdn.linear_prefill_workspace_bytes(1, 4096, 4, 128, 128, dtype)
    assert need > 0
    assert gdn.linear_prefill_workspace_bytes(1, 1, 4, 128, 128, dtype) == 0
    assert gdn.linear_prefill_workspace_bytes(0, 4096, 4, 128, 128, dtype) == 0
    assert gdn.linear_prefill_workspace_bytes(3, 0, 4, 128, 128, dtype) == 0
    for kw in (dict(ws=None), dict(ws_bytes=need - 1), dict(ws=P + 8), dict(ws=P, ws_bytes=0)):
        assert _c_prefill(lib, dtype=code, total_T=4096, **{"ws_bytes": need, **kw}) == INV
        assert "workspace" in lib.gdn_last_error().decode()


@pytest.mark.parametrize("name", ["gdn_linear_decode", "gdn_linear_decode_bf16_state"])
@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INV), (dict(state=None), INV), (dict(Hv=5), INV), (dict(B=-1), INV), (dict(dk=100), UNS),
    (dict(dtype=3), INV), (dict(state=P + 4), INV), (dict(g=P + 1), INV), (dict(g_stride=2), INV),
    (dict(B=1 << 30), INV),
], ids=str)
def test_decode_refuses(lib, name, kw, status):
    assert _c_decode(lib, name, **kw) == status
    assert lib.gdn_last_error().decode().startswith(name)


def test_empty_problems_are_no_ops(lib):
    assert _c_prefill(lib, n_seqs=0, q=None, k=None, v=None, o=None, cu=None, state_out=None) == gdn.GDN_OK
    assert _c_decode(lib, B=0, q=None, state=None, o=None) == gdn.GDN_OK
    assert lib.gdn_last_error() == b""


def test_the_binding_wants_cuda_tensors():
    z = torch.zeros(4, 2, 128, dtype=BF16)
    with pytest.raises(TypeError):
        gdn.linear_prefill(z, z, z, torch.zeros(4, 2))
    with pytest.raises(TypeError):
        gdn.linear_decode(z, z, z, torch.zeros(4, 2), torch.zeros(4, 2, 128, 128))


@pytest.mark.gpu
def test_the_binding_checks_shapes_types_and_layout():
    x = on_gpu(draw([20, 12], 2, 4, 128, 128, BF16, seed=40))
    call = lambda **kw: (lambda a: gdn.linear_prefill(a["q"], a["k"], a["v"], a["g"], a["state_in"], a["cu"],  # noqa: E731
                                                       **{n: a[n] for n in a if n in ("o", "state_out")}))({**x, **kw})
    for kw, err in ((dict(k=x["k"][:31]), ValueError), (dict(k=x["k"].half()), TypeError), (dict(g=x["g"].half()), TypeError),
                    (dict(g=x["g"][:, :3].contiguous()), ValueError), (dict(g=x["g"].t().contiguous().t()), ValueError),
                    (dict(state_in=x["state_in"].to(BF16)), TypeError), (dict(state_in=x["state_in"][:1]), ValueError),
                    (dict(cu=x["cu"].long()), TypeError), (dict(cu=x["cu"][:0]), ValueError), (dict(cu=x["cu"].cpu()), TypeError),
                    (dict(q=x["q"].double(), k=x["k"].double(), v=x["v"].double()), TypeError),
                    (dict(o=torch.empty(31, 4, 128, dtype=BF16, device=DEV)), ValueError),
                    (dict(state_out=torch.empty(2, 4, 128, 128, dtype=BF16, device=DEV)), TypeError),
                    (dict(q=x["q"].view(32, 256)), ValueError)):
        with pytest.raises(err):
            call(**kw)
    s = x["state_in"]
    with pytest.raises(ValueError):
        gdn.linear_decode(x["q"][:2], x["k"][:2], x["v"][:2], x["g"][:2], s[:1])
    with pytest.raises(TypeError):
        gdn.linear_decode(x["q"][:2], x["k"][:2], x["v"][:2], x["g"][:2], s.half())
    with pytest.raises(gdn.GdnError):
        big = torch.zeros(2, 1, 256, dtype=BF16, device=DEV)
        gdn.linear_decode(big, big, big, torch.zeros(2, 1, device=DEV), torch.zeros(2, 1, 256, 256, device=DEV))
