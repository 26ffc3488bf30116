"""Decayed linear attention at values and calls where it could go wrong: tokens of
unlike size in one block, and what follows below. References and bounds are those
of tests/_linear_ref.py.
"""
import os
import re
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from tests import _linear_ref as ref
from tests.test_linear_attention import check, draw, prefill

gdn = pytest.importorskip("gated_deltanet_linear_21_b200")

DEV = "cuda"
CSRC = os.path.join(os.path.dirname(gdn.__file__), "csrc")
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


# ------------------------------------------ tokens of unlike size in a block ---

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("at", [0, 63, 100, 127, 200])
@pytest.mark.parametrize("grow,v", [(128, 0), (512, -8), (4096, -14)], ids=str)
def test_a_large_token_leaves_the_others_of_its_block_as_they_were(dtype, at, grow, v):
    """One token's q and k enlarged (its v small, so that every output stays in f16's
    range), in a block that decays by 18 bits: the other rows keep their precision."""
    x = draw([256], 1, 2, 128, 128, dtype, seed=70)
    x["g"] = torch.full((2,), -18 * 0.6931 / 128)
    for n in ("q", "k"):
        x[n][at] = (x[n][at].float() * grow).to(dtype)
    x["v"][at] = (x["v"][at].float() * 2.0 ** v).to(dtype)
    check(x, *prefill(x))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("g", [-5.0, -0.7, -0.05])
@pytest.mark.parametrize("dk", [128, 64])
def test_small_channels_of_k_keep_their_precision_in_the_state(dtype, g, dk):
    """Channels and tokens of k at powers of two from 2^-12 to 2^6, so that a channel's part of
    the state may come from products far below the block's largest."""
    x = draw([128, 300, 1, 140], 2, 2, dk, 64, dtype, seed=88)
    gen = torch.Generator().manual_seed(89)
    size = lambda *shape: torch.exp2(torch.randint(-6, 4, shape, generator=gen).float())  # noqa: E731
    x["k"] = (x["k"].float() * size(569, 1, 1) * size(1, 2, dk)).to(dtype)
    x["g"] = torch.full((2,), g)
    check(x, *prefill(x))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_far_tokens_keep_their_precision_in_the_state(dtype, seed):
    """Decays of e^-5 a token, tokens of k and v at powers of two from 2^-6 to 2^4: an element of
    the state may come from a token whose weight is 2^-30."""
    x = draw([300, 1, 128, 44, 20, 130], 2, 6, 128, 128, dtype, "strong", seed=90 + seed)
    gen = torch.Generator().manual_seed(91 + seed)
    for n in "kv":
        x[n] = (x[n].float() * torch.exp2(torch.randint(-6, 5, (623, x[n].shape[1], 1), generator=gen).float())).to(dtype)
    o, s = prefill(x)
    _, rs, _, ms = ref.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["state_in"], x["cu"])
    for n, T in enumerate([300, 1, 128, 44, 20, 130]):      # each sequence within its own bound
        ref.check_state(s[n], rs[n], ms[n], min(T, 64))     # (what is older than 64 tokens is gone)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("bits", [1, 18, 45, 100])
def test_rows_of_every_size_in_a_block(dtype, bits):
    """q and k of each token, and the state, at their own powers of two."""
    x = draw([300, 130], 2, 2, 128, 64, dtype, seed=71)
    gen = torch.Generator().manual_seed(72)
    size = lambda lo, hi, n: torch.exp2(torch.randint(lo, hi + 1, (n, 1, 1), generator=gen).float())  # noqa: E731
    x["q"] = (x["q"].float() * size(-12, 4, 430)).to(dtype)
    x["k"] = (x["k"].float() * size(-6, 4, 430)).to(dtype)
    x["state_in"][0] *= 2.0 ** 12
    x["state_in"][1] *= 2.0 ** -12
    x["g"] = torch.full((2,), -bits * 0.6931 / 128)
    o, s = prefill(x)
    ro, rs, mo, ms = ref.linear_prefill(x["q"], x["k"], x["v"], x["g"], x["state_in"], x["cu"])
    # rounding to nearest makes what is 65520 or more infinite in f16; the error before it is within 2^-10 mo
    near = np.abs(ro) + 2.0 ** -10 * mo >= 65520 if dtype == F16 else np.zeros(ro.shape, bool)
    got = ref.f64(o)
    assert (np.isfinite(got) | (near & (np.sign(got) == np.sign(ro)))).all()
    o = torch.where(torch.from_numpy(near & ~np.isfinite(got)).to(DEV), 0, o)
    ref.check_o(o, np.where(near & ~np.isfinite(got), 0, ro), mo, 300, 128)
    ref.check_state(s, rs, ms, 300)


# --------------------------------------------------- buffers that are used again ---

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lo,hi", [(1, 40), (100, 300)], ids=str)
def test_short_blocks_leave_their_buffers_to_the_next(dtype, lo, hi):
    """Many short blocks, whose o goes out through the buffer that a later Q comes into."""
    lengths = torch.randint(lo, hi + 1, (500,), generator=torch.Generator().manual_seed(73)).tolist()
    x = draw(lengths, 2, 4, 128, 128, dtype, seed=73)
    o, s = prefill(x)
    for _ in range(10):
        o2, s2 = prefill(x)
        assert torch.equal(o, o2) and torch.equal(s, s2)
    cu = x["cu"].tolist()
    for n in (0, 3, 250, 499):      # (the definition is slow)
        a, b = cu[n], cu[n + 1]
        y = dict(q=x["q"][a:b], k=x["k"][a:b], v=x["v"][a:b], g=x["g"][a:b], state_in=x["state_in"][n:n + 1],
                 cu=torch.tensor([0, b - a], dtype=torch.int32))
        check(y, o[a:b], s[n:n + 1])


# ----------------------------------------------------------------- bounded waits ---

@pytest.mark.gpu
def test_the_prefills_waits_end_by_themselves_and_the_context_survives():
    """The waits on chip, for a flag and of the scan, which nothing ends: the kernel returns
    within its limits (a timeout of the device; a check says that one did not end by itself)."""
    gdn.device_error()
    t0, t1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    t0.record()
    gdn.wait_selftest(2000)
    t1.record()
    with pytest.raises(gdn.GdnError) as err:
        gdn.device_error()
    assert err.value.status == gdn.GDN_ERR_DEVICE_TIMEOUT
    t1.synchronize()
    # two waits one after the other in the first kernel (2 ms each at 2 GHz), one in the second
    assert t0.elapsed_time(t1) > 5.0
    gdn.device_error()
    x = draw([1300, 40], 1, 2, 128, 128, BF16, seed=74)
    check(x, *prefill(x))


# ------------------------------------------------------------ one prompt, no offsets ---

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [0, 1, 200, 1500])
def test_one_prompt_without_cu_seqlens_captured_and_on_another_stream(dtype, T):
    x = draw([T], 1, 2, 128, 128, dtype, seed=76)
    d = {n: t.to(DEV) for n, t in x.items()}
    args = (d["q"], d["k"], d["v"], d["g"], d["state_in"])
    want = gdn.linear_prefill(*args, d["cu"])
    assert all(torch.equal(a, b) for a, b in zip(gdn.linear_prefill(*args), want))
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = gdn.linear_prefill(*args, stream=other)
    other.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gdn.linear_prefill(*args)
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    gdn.device_error()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T", [2500, 4096])
def test_errors_in_the_mean_square_with_a_slow_decay(dtype, T):
    """What bounds for single elements, which grow with T, let pass: a dropped term of K, or a
    decay that drifts. The state: at most 64 tokens (fp32) or 8 blocks in a row, then T / 64
    segments of two roundings, and the products' part as in the test above. o in 16 bits: its
    own rounding, at most u / sqrt(3) in the mean square, and independent of it the same of
    every term (one operand of each is rounded); in fp32 the state's, and of a sum of 128
    terms 12 roundings in a row (8 fma, 4 additions)."""
    x = draw([T], 1, 2, 128, 128, dtype, init=False, seed=86)
    x["g"] = torch.tensor([-3e-4, -2e-5])
    o, s = prefill(x)
    ro, rs, _, _ = ref.linear_prefill(x["q"], x["k"], x["v"], x["g"], None, x["cu"])
    rms = lambda got, want: np.sqrt(((ref.f64(got) - want) ** 2).mean((0, 2)) / (want ** 2).mean((0, 2))).max()  # noqa: E731
    state = rounded(64 * 17 / 16 + 2 * T / 64, False)
    if dtype != F32:
        state += 2.0 ** -23 * 16 / 12 ** 0.5 + 2 * 2.0 ** -22
    assert rms(s[0].transpose(0, 1), rs[0].transpose(1, 0, 2)) <= state      # [dv, heads, dk]
    u = torch.finfo(dtype).eps / 2
    assert rms(o, ro) <= (u * (2 / 3) ** 0.5 if dtype != F32 else state + rounded(12, False))


# ------------------------------------------------------------- infinities and NaN ---

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("what", ["v", "k", "q", "g"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("lengths", [[300, 40], [1400, 130]], ids=str)
def test_a_bad_token_reaches_what_the_definition_says(dtype, what, bad, lengths):
    """NaN and infinities in single channels: the rows before their token, and channels of
    v that they are not in, keep their values; all that depends on them is infinite or NaN."""
    if what == "g" and bad != bad or what == "g" and bad < 0:
        bad = float("nan")                                # (-inf is a reset, tested elsewhere)
    for at in ([(5, 0, 3), (130, 1, 70)], [(127, 1, 127), (128, 0, 0)], [(lengths[0] - 1, 0, 64), (lengths[0] + 30, 1, 9)],
               [(0, 0, 1), (lengths[0] // 2, 0, 2), (lengths[0] // 2 - 1, 1, 2)]):
        x = draw(lengths, 2, 2, 128, 128, dtype, seed=77)
        clean, poison = dict(x), dict(x)
        for y, z in ((x, bad), (clean, 0.0), (poison, float("nan"))):
            y[what] = y[what].clone()
            for t, h, c in at:
                y[what][(t, h, c)[:y[what].dim()]] = z
        o, s = prefill(x)
        reached = ref.linear_prefill(*(poison[n] for n in ("q", "k", "v", "g", "state_in", "cu")))[:2]
        ro, rs, mo, ms = ref.linear_prefill(*(clean[n] for n in ("q", "k", "v", "g", "state_in", "cu")))
        for got, mask, r, m, check_it in ((o, ~np.isfinite(reached[0]), ro, mo, lambda *a: ref.check_o(*a, max(lengths), 128)),
                                          (s, ~np.isfinite(reached[1]), rs, ms, lambda *a: ref.check_state(*a, max(lengths)))):
            mask_t = torch.from_numpy(mask).to(DEV)
            assert (mask.any() or (what == "q" and got is s)) and not torch.isfinite(got[mask_t]).any()
            check_it(got.masked_fill(mask_t, 0), np.where(mask, 0, r), np.where(mask, 0, m))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("dk,dv", [(128, 128), (16, 32), (64, 16)])
def test_many_bad_channels_with_the_state_in_place(dtype, dk, dv):
    """Rows in front of bad tokens are made again from the entering state, which the call
    overwrites: sequences of one segment and of several, every third channel bad."""
    lengths = [100, 1500, 0, 60, 200]
    x = draw(lengths, 1, 2, dk, dv, dtype, seed=78)
    cu = x["cu"].tolist()
    clean, poison = dict(x), dict(x)
    for y, z in ((x, float("inf")), (clean, 0.0), (poison, float("nan"))):
        y["v"] = y["v"].clone()
        for c in range(0, dv, 3):
            for n in (0, 1, 1, 4):
                y["v"][cu[n] + (37 * c + 11 * n) % lengths[n], c % 2, c] = z
            y["v"][cu[1] + 1030 + c, 1, c] = z
    d = {n: t.to(DEV) for n, t in x.items()}
    o = torch.full(x["v"].shape, 7.0, dtype=dtype, device=DEV)
    _, s = gdn.linear_prefill(d["q"], d["k"], d["v"], d["g"], d["state_in"], d["cu"], o=o, state_out=d["state_in"])
    gdn.device_error()
    reached = ref.linear_prefill(*(poison[n] for n in ("q", "k", "v", "g", "state_in", "cu")))[:2]
    ro, rs, mo, ms = ref.linear_prefill(*(clean[n] for n in ("q", "k", "v", "g", "state_in", "cu")))
    for got, mask, r, m, check_it in ((o, ~np.isfinite(reached[0]), ro, mo, lambda *a: ref.check_o(*a, 1500, dk)),
                                      (s, ~np.isfinite(reached[1]), rs, ms, lambda *a: ref.check_state(*a, 1500))):
        mask_t = torch.from_numpy(mask).to(DEV)
        assert mask.any() and not torch.isfinite(got[mask_t]).any()
        check_it(got.masked_fill(mask_t, 0), np.where(mask, 0, r), np.where(mask, 0, m))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("bad", [float("nan"), -float("inf")])
def test_a_bad_element_of_the_entering_state(dtype, bad):
    lengths = [1400, 0, 130]
    x = draw(lengths, 2, 2, 128, 128, dtype, seed=87)
    clean, poison = dict(x), dict(x)
    for y, z in ((x, bad), (clean, 0.0), (poison, float("nan"))):
        y["state_in"] = y["state_in"].clone()
        for at in ((0, 0, 5, 77), (0, 1, 100, 0), (1, 0, 3, 3), (2, 1, 127, 127)):
            y["state_in"][at] = z
    o, s = prefill(x)
    reached = ref.linear_prefill(*(poison[n] for n in ("q", "k", "v", "g", "state_in", "cu")))[:2]
    ro, rs, mo, ms = ref.linear_prefill(*(clean[n] for n in ("q", "k", "v", "g", "state_in", "cu")))
    for got, mask, r, m, check_it in ((o, ~np.isfinite(reached[0]), ro, mo, lambda *a: ref.check_o(*a, 1400, 128)),
                                      (s, ~np.isfinite(reached[1]), rs, ms, lambda *a: ref.check_state(*a, 1400))):
        mask_t = torch.from_numpy(mask).to(DEV)
        assert mask.any() and not torch.isfinite(got[mask_t]).any()
        check_it(got.masked_fill(mask_t, 0), np.where(mask, 0, r), np.where(mask, 0, m))


# ------------------------------------------------------------------ the debug build ---

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("lengths,Hqk,Hv", [([1], 1, 1), ([700, 0, 1500, 33], 2, 4), ([0, 3] * 60 + [1300], 2, 40)], ids=str)
def test_the_debug_build_checks_the_prefill_and_gives_the_same_bits(dtype, lengths, Hqk, Hv):
    lib = gdn.debug_lib()
    x = draw(lengths, Hqk, Hv, 64, 64, dtype, seed=79)
    want = prefill(x)
    d = {n: t.to(DEV) for n, t in x.items()}
    T, N = x["q"].shape[0], len(lengths)
    code = {BF16: gdn.GDN_BF16, F16: gdn.GDN_F16, F32: gdn.GDN_F32}[dtype]
    o, s = torch.full_like(want[0], 7.0), torch.full_like(want[1], 7.0)
    need = lib.gdn_linear_prefill_workspace_bytes(N, T, Hv, 64, 64, code)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    st = torch.cuda.current_stream().cuda_stream
    assert lib.gdn_linear_prefill(d["q"].data_ptr(), d["k"].data_ptr(), d["v"].data_ptr(), d["g"].data_ptr(), Hv,
                                  d["state_in"].data_ptr(), d["cu"].data_ptr(), N, T, Hqk, Hv, 64, 64, 0.0, code,
                                  o.data_ptr(), s.data_ptr(), ws.data_ptr(), need, st) == gdn.GDN_OK
    assert lib.gdn_device_error(st) == gdn.GDN_OK, lib.gdn_last_error().decode()
    assert torch.equal(o, want[0]) and torch.equal(s, want[1])


@pytest.mark.gpu
def test_the_debug_build_checks_the_pool():
    lib = gdn.debug_lib()
    x = torch.randn(5, 3, 128, 64, device=DEV)
    codes, exps = gdn.state_pool(4, 3, 128, 64)
    slots = torch.tensor([3, -1, 0, 9, 1], dtype=torch.int32, device=DEV)
    out, st = torch.empty_like(x), torch.cuda.current_stream().cuda_stream
    a = (slots.data_ptr(), 5, 4, 3, 64, 128, 0)
    assert lib.gdn_state_store(x.data_ptr(), gdn.GDN_F32, *a, codes.data_ptr(), exps.data_ptr(), st) == gdn.GDN_OK
    assert lib.gdn_state_load(codes.data_ptr(), exps.data_ptr(), *a, out.data_ptr(), gdn.GDN_F32, st) == gdn.GDN_OK
    assert lib.gdn_device_error(st) == gdn.GDN_OK, lib.gdn_last_error().decode()
    assert torch.equal(out, gdn.state_load(codes, exps, slots))


def test_the_kernels_hold_index_checks():
    """What the headers say of the debug build: a check in every kernel that works with indices from the device."""
    for name, kernels in (("linear_tc.cuh", 2), ("linear.cuh", 2), ("state_pool.cuh", 2)):
        assert open(os.path.join(CSRC, name)).read().count("GDN_CHECK(") >= kernels, name


# ------------------------------------------------------- many calls, few segments ---

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_last_segments_that_follow_one_another_on_a_cta(dtype):
    """Sequences of two segments, more of them than CTAs: a CTA's items are last ones in a row, whose
    flags come early. A wait that missed its turn would run out."""
    x = draw([1100, 1300] * 12, 4, 32, 128, 128, dtype, init=False, seed=85)
    d = {n: t.to(DEV) if t is not None else None for n, t in x.items()}
    state = torch.randn(24, 32, 128, 128, device=DEV)
    first = gdn.linear_prefill(d["q"], d["k"], d["v"], d["g"], state, d["cu"])
    for i in range(150):
        got = gdn.linear_prefill(d["q"], d["k"], d["v"], d["g"], state, d["cu"])
        if i % 10 == 0:
            assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
    gdn.device_error()


# ------------------------------------------------------------------- host threads ---

@pytest.mark.gpu
@pytest.mark.parametrize("name", ["linear_prefill", "prefill"])
def test_a_new_host_thread_calls_first(name):
    """A thread that has made no CUDA call yet, with every buffer given, so that nothing before the
    call makes the device's context the thread's."""
    x = draw([200], 1, 2, 128, 128, BF16, init=False, seed=95)
    d = {n: t.to(DEV) for n, t in x.items() if t is not None}
    beta = torch.full((200, 2), 0.5, device=DEV)
    o, s = torch.empty_like(d["v"]), torch.empty(1, 2, 128, 128, device=DEV)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
    args = (d["q"], d["k"], d["v"], d["g"]) + ((beta,) if name == "prefill" else ()) + (None, d["cu"])
    want = [t.clone() for t in getattr(gdn, name)(*args, o=o, state_out=s, workspace=ws)]
    torch.cuda.synchronize()
    failed = []

    def call():
        try:
            getattr(gdn, name)(*args, o=o, state_out=s, workspace=ws)
        except Exception as e:                # noqa: BLE001
            failed.append(e)

    for _ in range(20):
        o.zero_()
        s.zero_()
        torch.cuda.synchronize()
        t = threading.Thread(target=call)
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert not failed, failed
        assert torch.equal(o, want[0]) and torch.equal(s, want[1])


# ------------------------------------------------------- sizes that are refused ---

@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_workspace_of_sizes_that_are_not_supported(dtype):
    """In a process of its own: no such size may end it."""
    code = ("import torch, gated_deltanet_linear_21_b200 as gdn\n"
            "f = lambda *a: gdn.linear_prefill_workspace_bytes(*a, dtype=torch.%s)\n"
            "for dk, dv in ((128, 0), (0, 128), (0, 0), (128, -1), (128, -40), (96, 128), (128, 2 ** 31 - 1)):\n"
            "    assert f(1, 4096, 4, dk, dv) == 0, (dk, dv)\n"
            "assert f(1, 2 ** 31, 4, 128, 128) == 0 and f(1, 2 ** 62, 2 ** 31 - 1, 128, 128) == 0\n" % dtype)
    done = subprocess.run([sys.executable, "-c", code], cwd=os.path.dirname(os.path.dirname(gdn.__file__)),
                          capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, (done.returncode, done.stderr[-500:])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_heads_of_no_rows_are_refused(dtype):
    z = lambda *shape: torch.zeros(*shape, dtype=dtype, device=DEV)  # noqa: E731
    with pytest.raises(gdn.GdnError) as err:
        gdn.linear_prefill(z(64, 2, 128), z(64, 2, 128), z(64, 4, 0), torch.zeros(64, 4, device=DEV))
    assert err.value.status == gdn.GDN_ERR_UNSUPPORTED


# ------------------------------------------------- a cu_seqlens that breaks its rules ---

def guarded(shape, dtype, fill):
    """(tensor, its surroundings): a tensor inside a larger buffer of `fill`."""
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * 8192,), fill, dtype=dtype, device=DEV)
    return buf[8192:8192 + n].view(shape), (buf[:8192], buf[8192 + n:])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("cu", [[-5, 50, 4000], [90, 20, 120], [200, 300, 400], [0, 120, 0, 120], [0, 2 ** 31 - 1],
                                [-2 ** 31, 2 ** 31 - 1, 60], [120, 0]], ids=str)
def test_a_broken_cu_seqlens_leaves_what_surrounds_the_arrays(dtype, cu):
    T, Hqk, Hv, dk, dv = 120, 1, 2, 128, 128
    x = draw([T], Hqk, Hv, dk, dv, dtype, seed=75)
    N, fill = len(cu) - 1, 3.0
    arrays = [guarded(t.shape, t.dtype, fill) for t in (x["q"], x["k"], x["v"], x["g"])]
    for (t, _), n in zip(arrays, "qkvg"):
        t.copy_(x[n])
    arrays += [guarded((N, Hv, dv, dk), F32, fill), guarded(x["v"].shape, dtype, fill), guarded((N, Hv, dv, dk), F32, fill)]
    need = gdn.linear_prefill_workspace_bytes(N, T, Hv, dk, dv, dtype)
    ws, around = guarded((need,), torch.uint8, 171)
    q, k, v, g, s0, o, s = (t for t, _ in arrays)
    gdn.linear_prefill(q, k, v, g, s0, torch.tensor(cu, dtype=torch.int32, device=DEV), o=o, state_out=s, workspace=ws)
    gdn.device_error()
    for _, (a, b) in arrays:
        assert (a == fill).all() and (b == fill).all()
    assert (around[0] == 171).all() and (around[1] == 171).all()
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (g, "g")):
        assert torch.equal(t.cpu(), x[n])
    assert (s0 == fill).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_sequences_that_overlap_many_times(dtype):
    """Far more items than the arrays' sizes allow for; with longer arrays they would pass 2^31."""
    T, Hv, N = 20000, 8, 2000
    z = lambda *shape, t=dtype: torch.zeros(*shape, dtype=t, device=DEV)  # noqa: E731
    cu = torch.tensor([0, T] * N, dtype=torch.int32, device=DEV)
    ws = torch.full((gdn.linear_prefill_workspace_bytes(2 * N - 1, T, Hv, 16, 16, dtype) + 65536,), 171, dtype=torch.uint8, device=DEV)
    gdn.linear_prefill(z(T, 1, 16), z(T, 1, 16), z(T, Hv, 16), z(T, Hv, t=F32), None, cu, workspace=ws[:-65536])
    gdn.device_error()
    assert (ws[-65536:] == 171).all()


# ------------------------------------------------------------- decays carried far ---

def drift(lengths, Hv, dtype, seed, lo=-6.0, hi=-3.0):
    """Largest over heads and sequences of the state's error (root of the mean square, relative)
    with a slow decay fixed per head, where the same rounding comes back at every step. The
    definition in closed form: S = sum_t exp(g (T - 1 - t)) v_t k_t^T in 64 bits."""
    x = draw(lengths, 1, Hv, 16, 16, dtype, init=False, seed=seed)
    gen = torch.Generator().manual_seed(seed)
    x["g"] = -torch.pow(10.0, lo + (hi - lo) * torch.rand(Hv, generator=gen))
    _, s = prefill(x)
    got, k, v, g = ref.f64(s), ref.f64(x["k"])[:, 0], ref.f64(x["v"]), ref.f64(x["g"])
    worst = 0.0
    for n, T in enumerate(lengths):
        a = int(x["cu"][n])
        for h in range(Hv):
            w = np.exp(g[h] * np.arange(T - 1, -1, -1))
            want = (v[a:a + T, h] * w[:, None]).T @ k[a:a + T]
            worst = max(worst, np.sqrt(((got[n, h] - want) ** 2).mean() / (want ** 2).mean()))
    return worst


# A rounding of the state is at most half a step of 2^-23 relative, 2^-23 / sqrt(12) in the root
# of the mean square, and n of them in a row, independent, sqrt(n) times that; from a state that
# grows from zero as sqrt(t) the sum of their squares halves. 256 elements of a head: 1.25 is 4
# deviations.
def rounded(n, grows=True):
    return 1.25 * 2.0 ** -23 * (n / (24 if grows else 12)) ** 0.5


@pytest.mark.gpu
def test_fp32_decays_do_not_drift():
    # unsplit, every token and every 16 tokens a rounding
    assert drift([4096], 400, F32, 80) <= rounded(4096 * 17 / 16)
    # two long segments and a first pass
    assert drift([8000, 10, 10, 10], 400, F32, 81) <= rounded(8000 * 17 / 16)
    # many segments: 144 tokens in each, 694 of them, two roundings each
    for seed in range(82, 90):
        assert drift([100000], 1, F32, seed, lo=-7.0, hi=-5.0) <= rounded(144 * 17 / 16 + 2 * 694, False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_decays_do_not_drift_on_the_tensor_cores(dtype):
    """196 segments of 8 blocks: two roundings for each that the state passes, and each
    block's own part: its products, 4 terms x 8 steps added in fp32, each off by at most 2^-24 of
    what is there (2^-23 where the unit cuts off instead of rounding: 2^-23 x 32 / 2 on
    average over a growing sum, times 1 / sqrt(12) where the signs differ), the terms' 2^-22 and
    the weights' 2^-22."""
    own = 2.0 ** -23 * 16 / 12 ** 0.5 + 2 * 2.0 ** -22
    for seed in range(90, 98):
        assert drift([200000], 1, dtype, seed, lo=-7.0, hi=-5.0) <= rounded(2 * 196 + 8, False) + own


# ------------------------------------------------------------- the kernel's text ---

def test_a_group_of_four_warps_changes_its_registers_at_one_place():
    """setmaxnreg has to be one instruction for the four warps of a group; the roles of
    warps 8 to 11 part, so it stands before them. A run cannot show a breach."""
    text = open(os.path.join(CSRC, "linear_tc.cuh")).read()
    body = text[text.index("prefill_kernel("):]
    calls = [m.start() for m in re.finditer(r"\b(give|take)_registers\(\);", body)]
    assert len(calls) == 2
    assert re.search(r"if \(warp >= kLoadWarp\) {\s+(//.*\s+)?give_registers\(\);\s+if \(warp == kLoadWarp\) {", body)
    assert re.search(r"  } else {\s+take_registers\(\);.*\s+// -+ compute warps ---", body)


def test_rows_of_o_written_without_a_bulk_copy_are_fenced_too():
    """Both ways out of the buffer end in a proxy fence, before its next bulk load. A run
    hardly ever shows one that is missing."""
    text = open(os.path.join(CSRC, "linear_tc.cuh")).read()
    body = text[text.index("auto send_o = "):]
    body = body[:body.index("\n    };")]
    bulk, plain = body.split("} else {")
    assert "fence_async_smem();" in bulk and "fence_async_smem();" in plain
