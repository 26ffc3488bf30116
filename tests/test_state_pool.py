"""The 8-bit state pool (state_pool, state_store, state_load) against its
definition in 64 bits: scaling by powers of two is exact and the codes' rounding
is to nearest even, so every value and exponent byte has to be equal.
"""
import numpy as np
import pytest
import torch

from tests import _linear_ref as ref

gdn = pytest.importorskip("gated_deltanet_linear_21_b200")

DEV = "cuda"
P = 0x10000  # a 16-byte aligned fake device address (never dereferenced)
E4M3, I8 = torch.float8_e4m3fn, torch.int8
F32, BF16 = torch.float32, torch.bfloat16
CODES = [E4M3, I8]


def states(n, Hv, dv, dk, sdtype, seed=0):
    gen = torch.Generator().manual_seed(8000 + seed)
    x = torch.randn(n, Hv, dv, dk, generator=gen)
    return (x * torch.exp2(torch.randint(-40, 40, (n, Hv, dv, 1), generator=gen).float())).to(sdtype)


def same(a, b):
    a, b = np.asarray(a, dtype=np.float64), np.asarray(b, dtype=np.float64)
    return a.shape == b.shape and bool(((a == b) | (np.isnan(a) & np.isnan(b))).all())


def rounded(values, dtype):
    """64-bit values rounded to a state type."""
    return ref.f64(torch.from_numpy(values).to(dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("sdtype", [F32, BF16])
@pytest.mark.parametrize("n,slots,Hv,dv,dk", [(1, 1, 1, 16, 16), (3, 7, 2, 16, 32), (5, 5, 3, 64, 64), (4, 9, 2, 128, 128),
                                              (2, 2, 5, 32, 16), (1, 3, 17, 128, 128)])
def test_store_and_load(code, sdtype, n, slots, Hv, dv, dk):
    x = states(n, Hv, dv, dk, sdtype)
    slot = torch.randperm(slots, generator=torch.Generator().manual_seed(1))[:n].to(torch.int32)
    codes, exps = gdn.state_pool(slots, Hv, dv, dk, dtype=code)
    assert exps.shape == (slots, Hv, dv, max(1, dk // 32))
    gdn.state_store(x.to(DEV), codes, exps, slot.to(DEV))
    val, e = ref.quantise(x, code)
    assert np.array_equal(exps.cpu().numpy()[slot.numpy()], e)
    out = torch.full((n, Hv, dv, dk), float("nan"), dtype=sdtype, device=DEV)
    assert gdn.state_load(codes, exps, slot.to(DEV), state=out) is out
    assert same(ref.f64(out), rounded(val, sdtype))
    # the other type reads the same codes, and slots nobody stored are zero states
    other = BF16 if sdtype == F32 else F32
    assert same(ref.f64(gdn.state_load(codes, exps, slot.to(DEV), dtype=other)), rounded(val, other))
    free = sorted(set(range(slots)) - set(slot.tolist()))
    if free:
        assert (gdn.state_load(codes, exps, torch.tensor(free, dtype=torch.int32, device=DEV)) == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
def test_rounding_at_every_border(code):
    """Every code, every midpoint between two codes and its neighbours, at several exponents."""
    if code == E4M3:
        grid = torch.arange(0, 127).to(torch.uint8).view(E4M3).double()      # 0 .. 448
    else:
        grid = torch.arange(0, 128).double()
    mid = (grid[1:] + grid[:-1]) / 2
    pts = torch.cat([grid, mid, mid * (1 + 2.0 ** -23), mid * (1 - 2.0 ** -24)]).float()
    pts = torch.cat([pts, -pts])
    top = float(grid[-1])
    rows = torch.zeros(-(-pts.numel() // 31), 32)
    rows[:, 0] = top                                                          # pins the group's exponent
    body = torch.zeros(rows.shape[0] * 31)
    body[: pts.numel()] = pts
    rows[:, 1:] = body.view(-1, 31)
    rows = torch.cat([rows * 2.0 ** e for e in (0, -100, 80, -117)])
    pad = -rows.shape[0] % 16
    x = torch.cat([rows, torch.zeros(pad, 32)]).view(1, -1, 16, 32)
    codes, exps = gdn.state_pool(1, x.shape[1], 16, 32, dtype=code)
    slot = torch.zeros(1, dtype=torch.int32, device=DEV)
    gdn.state_store(x.to(DEV), codes, exps, slot)
    val, e = ref.quantise(x, code)
    assert np.array_equal(exps.cpu().numpy(), e)
    assert same(ref.f64(gdn.state_load(codes, exps, slot)), val)


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("sdtype", [F32, BF16])
def test_extremes(code, sdtype):
    big = torch.finfo(sdtype).max
    x = torch.zeros(1, 1, 16, 64, dtype=sdtype)
    x[0, 0, 0, 3] = big
    x[0, 0, 0, 40] = -big
    x[0, 0, 1, 5] = torch.finfo(sdtype).tiny                     # the smallest normal number
    x[0, 0, 2, 7] = float("inf")
    x[0, 0, 3, 33] = float("nan")
    x[0, 0, 4, 1] = -float("inf")
    x[0, 0, 5] = 448.0
    x[0, 0, 6, :32] = 448.0
    x[0, 0, 6, 0] = 450.0
    x[0, 0, 7] = 127.0
    x[0, 0, 8, 0] = -127.5
    x[0, 0, 9] = -0.0
    x[0, 0, 10] = torch.finfo(sdtype).tiny / 8                   # a subnormal
    x[0, 0, 11, ::2] = 2.0 ** -126
    x[0, 0, 11, 1] = 2.0 ** -120
    codes, exps = gdn.state_pool(1, 1, 16, 64, dtype=code)
    slot = torch.zeros(1, dtype=torch.int32, device=DEV)
    gdn.state_store(x.to(DEV), codes, exps, slot)
    val, e = ref.quantise(x, code)
    assert np.array_equal(exps.cpu().numpy(), e)
    assert same(ref.f64(gdn.state_load(codes, exps, slot)), rounded(val, F32))
    assert same(ref.f64(gdn.state_load(codes, exps, slot, dtype=BF16)), rounded(rounded(val, F32), BF16))


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
def test_storing_what_was_loaded_keeps_the_values(code):
    x = states(6, 4, 128, 128, F32, seed=3).to(DEV)
    codes, exps = gdn.state_pool(6, 4, 128, 128, dtype=code)
    slot = torch.arange(6, dtype=torch.int32, device=DEV)
    gdn.state_store(x, codes, exps, slot)
    once = gdn.state_load(codes, exps, slot)
    for _ in range(3):
        gdn.state_store(gdn.state_load(codes, exps, slot), codes, exps, slot)
    assert torch.equal(gdn.state_load(codes, exps, slot), once)


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
def test_slots_outside_the_pool_and_slots_named_twice(code):
    x = states(700, 1, 16, 16, F32, seed=4)
    slots = 40
    gen = torch.Generator().manual_seed(5)
    slot = torch.randint(-3, slots + 3, (700,), generator=gen).to(torch.int32)
    slot[::50] = torch.iinfo(torch.int32).min
    slot[1::50] = torch.iinfo(torch.int32).max
    slot[slot == 11] = 12                                         # nobody's slot
    codes, exps = gdn.state_pool(slots, 1, 16, 16, dtype=code)
    exps[11], codes.view(torch.int8)[11] = 77, 5
    for _ in range(3):
        gdn.state_store(x.to(DEV), codes, exps, slot.to(DEV))
    assert (exps[11] == 77).all() and (codes.view(torch.int8)[11] == 5).all()
    val, _ = ref.quantise(x, code)
    out = ref.f64(gdn.state_load(codes, exps, slot.to(DEV)))
    last = {int(s): i for i, s in enumerate(slot.tolist())}
    for i, s in enumerate(slot.tolist()):
        assert same(out[i], val[last[s]] if 0 <= s < slots else np.zeros_like(out[i]))


@pytest.mark.gpu
def test_an_empty_pool_and_no_states():
    codes, exps = gdn.state_pool(0, 2, 16, 16)
    slot = torch.zeros(3, dtype=torch.int32, device=DEV)
    x = torch.ones(3, 2, 16, 16, device=DEV)
    gdn.state_store(x, codes, exps, slot)
    assert (gdn.state_load(codes, exps, slot) == 0).all()
    codes, exps = gdn.state_pool(2, 2, 16, 16)
    gdn.state_store(x[:0], codes, exps, slot[:0])
    assert gdn.state_load(codes, exps, slot[:0]).shape == (0, 2, 16, 16)


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
def test_a_pool_beyond_32_bit_offsets(code):
    slots, Hv, d = 1030, 128, 128
    x = states(2, Hv, d, d, F32, seed=10)
    codes, exps = gdn.state_pool(slots, Hv, d, d, dtype=code)
    assert codes.numel() > 2 ** 31
    slot = torch.tensor([slots - 1, 1023], dtype=torch.int32, device=DEV)
    gdn.state_store(x.to(DEV), codes, exps, slot)
    assert same(ref.f64(gdn.state_load(codes, exps, slot)), ref.quantise(x, code)[0])
    near = torch.tensor([0, 1022, 1024, slots - 2], dtype=torch.int32, device=DEV)
    assert not gdn.state_load(codes, exps, near).any()


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    x = states(4, 2, 128, 128, F32, seed=6).to(DEV)
    codes, exps = gdn.state_pool(6, 2, 128, 128)
    slot = torch.tensor([5, 0, 3, 2], dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.state_store(x, codes, exps, slot)
        out = gdn.state_load(codes, exps, slot)
    for seed in (7, 8):
        x.copy_(states(4, 2, 128, 128, F32, seed=seed))
        slot.copy_(torch.randperm(6)[:4])
        graph.replay()
        torch.cuda.synchronize()
        assert same(ref.f64(out), ref.quantise(x, E4M3)[0])
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    again = gdn.state_load(codes, exps, slot, stream=other)
    other.synchronize()
    assert torch.equal(again, out)


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
def test_a_conversation_set_aside_and_resumed(code):
    """Prompt, states set aside, resumed in another order and number, the prompts continued, then decoded."""
    gen = torch.Generator().manual_seed(9)
    Hqk, Hv, d = 2, 4, 128
    first, second = [150, 40, 0, 300], [70, 1, 129]
    rnd = lambda n, h: torch.randn(n, h, d, generator=gen).to(BF16)  # noqa: E731
    decay = lambda n: torch.nn.functional.logsigmoid(torch.randn(n, Hv, generator=gen) + 3)  # noqa: E731
    a = [rnd(sum(first), Hqk), rnd(sum(first), Hqk), rnd(sum(first), Hv), decay(sum(first))]
    b = [rnd(sum(second), Hqk), rnd(sum(second), Hqk), rnd(sum(second), Hv), decay(sum(second))]
    cu = lambda ls: torch.tensor([0] + ls).cumsum(0).to(torch.int32)  # noqa: E731
    dev = lambda ts: [t.to(DEV) for t in ts]  # noqa: E731
    _, s1 = gdn.linear_prefill(*dev(a), None, cu(first).to(DEV))
    codes, exps = gdn.state_pool(5, Hv, d, d, dtype=code)
    gdn.state_store(s1, codes, exps, torch.tensor([4, 1, 0, 2], dtype=torch.int32, device=DEV))
    back = torch.tensor([2, -1, 4], dtype=torch.int32, device=DEV)       # the last, a new one, the first
    s2 = gdn.state_load(codes, exps, back)
    want = ref.quantise(s1, code)[0]
    want = np.stack([want[3], np.zeros_like(want[0]), want[0]])
    assert same(ref.f64(s2), want)
    o, s3 = gdn.linear_prefill(*dev(b), s2, cu(second).to(DEV), state_out=s2)
    ro, rs, mo, ms = ref.linear_prefill(*b, torch.from_numpy(want), cu(second))
    ref.check_o(o, ro, mo, 129, d)
    ref.check_state(s3, rs, ms, 129)
    c = [rnd(3, Hqk), rnd(3, Hqk), rnd(3, Hv), decay(3)]
    before = s3.cpu()
    o = gdn.linear_decode(*dev(c), s3)
    ro, rs, mo, ms = ref.linear_prefill(*c, before, range(4))
    ref.check_o(o, ro, mo, 1, d)
    ref.check_state(s3, rs, ms, 1)
    gdn.device_error()


@pytest.mark.gpu
def test_the_pool_serves_the_gated_delta_rule_too():
    import workloads
    x = workloads.prefill_inputs([90, 33], Hqk=2, Hv=4, d=128, seed=5, state_std=0.05)
    d = {n: t.to(DEV) if isinstance(t, torch.Tensor) else t for n, t in x.items()}
    _, s = gdn.prefill(d["q"], d["k"], d["v"], d["g"], d["beta"], d["state_in"], d["cu_seqlens"])
    codes, exps = gdn.state_pool(3, 4, 128, 128)
    slot = torch.tensor([2, 0], dtype=torch.int32, device=DEV)
    gdn.state_store(s, codes, exps, slot)
    state = gdn.state_load(codes, exps, slot)
    assert same(ref.f64(state), ref.quantise(s, E4M3)[0])
    o = gdn.decode(d["q"][:2], d["k"][:2], d["v"][:2], d["g"][:2], d["beta"][:2], state)
    assert torch.isfinite(o.float()).all()


# ---------------------------------------------------------------- refusals ---
INV, UNS = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_linear_21_b200 import build as gdn_build
    gdn_build.build()
    return gdn.lib()


def _store(lib, **kw):
    a = dict(state=P, sdt=gdn.GDN_F32, slots=P, n=2, n_slots=4, Hv=2, dk=128, dv=128, code=0, codes=P, exps=P, stream=None)
    a.update(kw)
    return lib.gdn_state_store(*a.values())


def _load(lib, **kw):
    a = dict(codes=P, exps=P, slots=P, n=2, n_slots=4, Hv=2, dk=128, dv=128, code=0, state=P, sdt=gdn.GDN_F32, stream=None)
    a.update(kw)
    return lib.gdn_state_load(*a.values())


@pytest.mark.parametrize("fn,name", [(_store, "gdn_state_store"), (_load, "gdn_state_load")])
@pytest.mark.parametrize("kw,status", [
    (dict(state=None), INV), (dict(slots=None), INV), (dict(codes=None), INV), (dict(exps=None), INV), (dict(n=-1), INV),
    (dict(n_slots=-1), INV), (dict(Hv=0), INV), (dict(dk=48), UNS), (dict(dv=256), UNS), (dict(code=2), INV),
    (dict(sdt=gdn.GDN_F16), INV), (dict(sdt=9), INV), (dict(state=P + 8), INV), (dict(codes=P + 4), INV),
    (dict(slots=P + 2), INV), (dict(n=1 << 30, Hv=1 << 10), INV),
], ids=str)
def test_refusals(lib, fn, name, kw, status):
    assert fn(lib, **kw) == status
    assert lib.gdn_last_error().decode().startswith(name)


def test_no_states_is_a_no_op(lib):
    assert _store(lib, n=0, state=None, slots=None) == gdn.GDN_OK
    assert _load(lib, n=0, state=None, slots=None) == gdn.GDN_OK


def test_the_binding_refuses():
    with pytest.raises(TypeError):
        gdn.state_pool(2, 2, 16, 16, dtype=torch.uint8, device="cpu")
    for dv, dk in ((16, 0), (16, 96), (256, 16)):
        with pytest.raises(ValueError):
            gdn.state_pool(2, 2, dv, dk, device="cpu")
    codes, exps = gdn.state_pool(2, 2, 16, 16, device="cpu")
    with pytest.raises(TypeError):
        gdn.state_store(torch.zeros(1, 2, 16, 16), codes, exps, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        gdn.state_load(codes, exps, torch.zeros(1, dtype=torch.int32))


@pytest.mark.gpu
def test_the_binding_checks_shapes_types_and_layout():
    codes, exps = gdn.state_pool(4, 2, 16, 32)
    x = torch.zeros(2, 2, 16, 32, device=DEV)
    slot = torch.zeros(2, dtype=torch.int32, device=DEV)
    for args, err in (((x.half(), codes, exps, slot), TypeError), ((x, codes, exps, slot.long()), TypeError),
                      ((x[:1], codes, exps, slot), ValueError), ((x, codes, exps[:3], slot), ValueError),
                      ((x, codes.view(torch.uint8), exps, slot), TypeError), ((x, codes, exps.float(), slot), TypeError),
                      ((x.transpose(2, 3), codes, exps, slot), ValueError), ((x, codes, exps, slot[:1]), ValueError)):
        with pytest.raises(err):
            gdn.state_store(*args)
    with pytest.raises(ValueError):
        gdn.state_load(codes, exps, slot, state=x[:1])
    with pytest.raises(TypeError):
        gdn.state_load(codes, exps, slot, dtype=torch.float16)
