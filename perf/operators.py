"""What is measured of the decayed linear attention and of the quantised state pool.

Four operators, each through the package's public entry points (``own``) and in
a plain form of elementary torch operations:

  linear_prefill   S_t = exp(g_t) S_{t-1} + v_t k_t^T,  o_t = scale S_t q_t  over packed prompts
  linear_decode    one step of the same recurrence for every sequence of a batch, the state updated in place
  state_store      states -> 8-bit codes with one power-of-two exponent for each 32 values along d_k, by slot
  state_load       the codes read back, by slot

A case is a dict of plain values; ``op`` is "prefill", "decode", "park" (states
stored into their slots and read back, as for a sequence that is set aside and
resumed) or "load" (states of cached prefixes read for a new batch).
"""
import math

import numpy as np
import torch

own = False
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CHUNK = 128      # tokens the plain prefill takes at a time
QMAX = {"e4m3": 448.0, "i8": 127.0}


# ------------------------------------------------------------------- cases ---
def _prefill(name, n, lo, hi, hqk, hv, dk=128, dv=128, dtype="bf16", fixed=False, init=False, lseed=0):
    c = {"op": "prefill", "n": n, "lo": lo, "hi": hi, "hqk": hqk, "hv": hv, "dk": dk, "dv": dv, "dtype": dtype,
         "fixed": fixed, "init": init, "lseed": lseed}
    return dict(c, name=name) if name else c


def _decode(name, b, hqk, hv, d=128, dtype="bf16", sdtype="f32", fixed=False):
    c = {"op": "decode", "b": b, "hqk": hqk, "hv": hv, "dk": d, "dv": d, "dtype": dtype, "sdtype": sdtype, "fixed": fixed}
    return dict(c, name=name) if name else c


def _cache(name, op, n, slots, hv, d=128, sdtype="f32", fmt="e4m3"):
    c = {"op": op, "n": n, "slots": slots, "hv": hv, "dk": d, "dv": d, "sdtype": sdtype, "fmt": fmt}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one short question: latency
        _prefill("prefill_77_h16", 1, 77, 77, 16, 16),
        # the benchmark's prompt
        _prefill("prefill_4096_h16", 1, 4096, 4096, 16, 16),
        # the benchmark's packed batch, continued from cached states
        _prefill("prefill_packed8_h32", 8, 128, 8192, 16, 32, init=True, lseed=5005),
        # many short requests packed in one call
        _prefill("prefill_packed64_h32", 64, 20, 300, 16, 32, lseed=7),
        # the benchmark's long prompt, in f16, a fixed decay for each head
        _prefill("prefill_32768_h32_f16", 1, 32768, 32768, 16, 32, dtype="f16", fixed=True),
        # fp32 inputs, small heads
        _prefill("prefill_f32_d64", 2, 500, 2000, 8, 16, dk=64, dv=64, dtype="f32", lseed=3),
        # a single conversation's step: latency
        _decode("decode_b1_h16", 1, 16, 16),
        # the benchmark's batch
        _decode("decode_b64_h32", 64, 16, 32),
        # an odd batch with states kept in bf16
        _decode("decode_b131_h32_s16", 131, 16, 32, dtype="f16", sdtype="bf16", fixed=True),
        # a batch of the benchmark's sequences set aside and resumed
        _cache("park_64_h32_e4m3", "park", 64, 80, 32),
        # a few sequences whose states are kept in bf16, as integers
        _cache("park_5_h16_i8", "park", 5, 9, 16, sdtype="bf16", fmt="i8"),
        # a new batch starts from cached prefixes
        _cache("load_48_h32_e4m3", "load", 48, 96, 32),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "decode", "decode", "park", "load"])
    hqk, hv = rng.choice([(4, 4), (2, 8), (8, 8), (16, 16), (8, 16), (16, 32), (32, 32)])
    if op == "prefill":
        n = _spread(rng, 1, 48)
        mean = _spread(rng, 16, max(17, min(32768 // n, 32768 * 16 // (n * hv))))
        lo = rng.randint(1, mean)
        plain16 = rng.random() < 0.7
        return _prefill(None, n, lo, 2 * mean - lo, hqk, hv,
                        dk=128 if plain16 else rng.choice([16, 32, 64, 128]), dv=128 if plain16 else rng.choice([16, 32, 64, 128]),
                        dtype=rng.choice(["bf16", "bf16", "f16"]) if plain16 else rng.choice(["bf16", "f16", "f32"]),
                        fixed=rng.random() < 0.3, init=rng.random() < 0.5, lseed=rng.randrange(1 << 20))
    if op == "decode":
        return _decode(None, _spread(rng, 1, 160), hqk, hv, d=rng.choice([64, 128, 128]), dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                       sdtype=rng.choice(["f32", "f32", "bf16"]), fixed=rng.random() < 0.3)
    n = _spread(rng, 1, 64)
    return _cache(None, op, n, n + rng.randint(0, 40), hv, d=rng.choice([64, 128, 128]), sdtype=rng.choice(["f32", "bf16"]),
                  fmt=rng.choice(["e4m3", "e4m3", "i8"]))


def _lengths(c):
    r = np.random.RandomState(c["lseed"])
    return [int(x) for x in r.randint(c["lo"], c["hi"] + 1, c["n"])]


# ------------------------------------------------------------------ inputs ---
def _decay(gen, rows, hv, fixed):
    """Log-decays: fixed ones of 1 - 2^-5 .. 1 - 2^-11 over the heads, or log sigmoid of N(3, 1) for each token."""
    if fixed:
        h = torch.arange(hv, device=DEV, dtype=torch.float64)
        jitter = torch.rand(hv, generator=gen, device=DEV, dtype=torch.float64)
        return torch.log1p(-torch.exp2(-5 - 6 * (h + jitter) / hv)).float()
    x = torch.randn(rows, hv, generator=gen, device=DEV, dtype=torch.float64) + 3
    return torch.nn.functional.logsigmoid(x).float()


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *shape: torch.randn(*shape, generator=gen, device=DEV)  # noqa: E731
    if c["op"] == "prefill":
        lens = _lengths(c)
        T, ty = sum(lens), TYPES[c["dtype"]]
        c["lens"] = lens
        c["cu"] = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
        c["q"], c["k"] = rn(T, c["hqk"], c["dk"]).to(ty), rn(T, c["hqk"], c["dk"]).to(ty)
        c["v"] = rn(T, c["hv"], c["dv"]).to(ty)
        c["g"] = _decay(gen, T, c["hv"], c["fixed"])
        c["state_in"] = rn(c["n"], c["hv"], c["dv"], c["dk"]) if c["init"] else None
    elif c["op"] == "decode":
        ty = TYPES[c["dtype"]]
        c["q"], c["k"] = rn(c["b"], c["hqk"], c["dk"]).to(ty), rn(c["b"], c["hqk"], c["dk"]).to(ty)
        c["v"] = rn(c["b"], c["hv"], c["dv"]).to(ty)
        c["g"] = _decay(gen, c["b"], c["hv"], c["fixed"])
        c["state"] = rn(c["b"], c["hv"], c["dv"], c["dk"]).to(TYPES[c["sdtype"]])
    else:
        group = min(32, c["dk"])
        shape = (c["slots"], c["hv"], c["dv"], c["dk"])
        c["slot"] = torch.randperm(c["slots"], generator=gen, device=DEV)[: c["n"]].to(torch.int32)
        if c["op"] == "park":
            spread = torch.exp(rn(c["n"], c["hv"], 1, 1))      # states of heads differ in size
            c["state"] = (rn(c["n"], *shape[1:]) * spread).to(TYPES[c["sdtype"]])
            c["codes"] = torch.zeros(shape, dtype=torch.int8, device=DEV)
            c["exps"] = torch.zeros(*shape[:-1], c["dk"] // group, dtype=torch.uint8, device=DEV)
        else:
            x = rn(*shape)
            c["codes"], c["exps"] = _quantise(x, c["fmt"])
        if c["fmt"] == "e4m3":
            c["codes"] = c["codes"].view(torch.float8_e4m3fn)
        c["out"] = torch.empty(c["n"], *shape[1:], dtype=TYPES[c["sdtype"]], device=DEV)
    return c


# ------------------------------------------------------------- plain forms ---
def _chunks(lens):
    """Token numbers [chunks, CHUNK] of the packed sequences' chunks, which of them are real, and each chunk's sequence."""
    n = torch.tensor(lens, device=DEV)
    start = n.cumsum(0) - n
    per = (n + CHUNK - 1) // CHUNK
    total = sum(-(-x // CHUNK) for x in lens)
    seq = torch.repeat_interleave(torch.arange(len(lens), device=DEV), per, output_size=total)
    first = per.cumsum(0) - per
    at = (torch.arange(total, device=DEV) - first[seq])[:, None] * CHUNK + torch.arange(CHUNK, device=DEV)
    real = at < n[seq][:, None]
    return torch.where(real, at + start[seq][:, None], 0), real, seq


def _plain_prefill(c):
    q, k, v, g, hv, dk = c["q"], c["k"], c["v"], c["g"], c["hv"], c["dk"]
    T, group = v.shape[0], hv // c["hqk"]
    out = torch.empty(T, hv, c["dv"], dtype=v.dtype, device=DEV)
    at, real, seq = _chunks(c["lens"])
    heads = lambda x: x[at].float().masked_fill(~real[..., None, None], 0).permute(0, 2, 1, 3)  # noqa: E731
    qc = heads(q).repeat_interleave(group, 1) * dk ** -0.5
    kc, vc = heads(k).repeat_interleave(group, 1), heads(v)
    gt = g.expand(T, hv) if g.dim() == 1 else g
    # log-decays summed in 64 bits within each chunk
    G = gt[at].double().masked_fill(~real[..., None], 0).permute(0, 2, 1).cumsum(-1)          # [chunks, hv, CHUNK]
    end = G[..., -1]
    # each chunk's own part of the state, and what every chunk finds when it begins
    U = (vc * (end[..., None] - G).exp().float()[..., None]).transpose(-1, -2) @ kc           # [chunks, hv, dv, dk]
    done = end.cumsum(0)
    N = c["n"]
    ones = torch.zeros(N, hv, dtype=torch.float64, device=DEV)
    total = ones.index_add(0, seq, end)
    before = (total.cumsum(0) - total)[seq]                                                    # decay of the sequences in front
    into, same = done - end - before, seq[:, None] == seq[None, :]
    order = torch.arange(len(seq), device=DEV)
    W = (into[:, None] - (done - before)[None, :]).masked_fill(~(same & (order[:, None] > order[None, :]))[..., None], -math.inf).exp().float()
    S = torch.matmul(W.permute(2, 0, 1), U.permute(1, 0, 2, 3).flatten(2)).view(hv, len(seq), c["dv"], dk).transpose(0, 1)
    Wn = (total[:, None] - (done - before)[None, :]).masked_fill(~(torch.arange(N, device=DEV)[:, None] == seq[None, :])[..., None], -math.inf).exp().float()
    state = torch.matmul(Wn.permute(2, 0, 1), U.permute(1, 0, 2, 3).flatten(2)).view(hv, N, c["dv"], dk).transpose(0, 1)
    if c["state_in"] is not None:
        S = S + into.exp().float()[..., None, None] * c["state_in"][seq]
        state = state + total.exp().float()[..., None, None] * c["state_in"]
    del U
    P = qc @ kc.transpose(-1, -2)
    P = P * (G[..., :, None] - G[..., None, :]).masked_fill(~torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV).tril(), -math.inf).exp().float()
    o = P @ vc + G.exp().float()[..., None] * (qc @ S.transpose(-1, -2))
    out[at[real]] = o.permute(0, 2, 1, 3)[real].to(v.dtype)
    return out, state.contiguous()


def _plain_decode(c):
    group = c["hv"] // c["hqk"]
    q, k = (c[x].float().repeat_interleave(group, 1) for x in ("q", "k"))
    S = c["g"].exp()[..., None, None] * c["state"].float() + c["v"].float()[..., None] * k[:, :, None, :]
    o = (S * q[:, :, None, :]).sum(-1) * c["dk"] ** -0.5
    c["state"].copy_(S)
    return o.to(c["v"].dtype), c["state"]


def _pow2(e):
    """2^e in 64 bits, exactly (exp2 and pow may be one unit off)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _quantise(x, fmt):
    """Codes (as bytes) and exponent bytes of x: for each group of 32 values the smallest e with max |x| <= QMAX 2^e."""
    group = min(32, x.shape[-1])
    y = x.double().unflatten(-1, (-1, group))
    m, e = torch.frexp(y.abs().amax(-1) / QMAX[fmt])
    e = torch.where(m == 0.5, e - 1, e).clamp(-127, 127)
    y = (y * _pow2(-e)[..., None]).flatten(-2).float()
    codes = y.to(torch.float8_e4m3fn).view(torch.int8) if fmt == "e4m3" else torch.round(y).to(torch.int8)
    return codes, (torch.where(m == 0, -127, e) + 127).to(torch.uint8)


def _plain_load(c):
    codes = c["codes"][c["slot"].long()] if c["fmt"] == "i8" else c["codes"].view(torch.int8)[c["slot"].long()].view(torch.float8_e4m3fn)
    e = c["exps"][c["slot"].long()].long() - 127
    return (codes.float().unflatten(-1, (e.shape[-1], -1)) * _pow2(e).float()[..., None]).flatten(-2).to(TYPES[c["sdtype"]])


def run(state):
    c = state
    if own:
        import gated_deltanet_linear_21_b200 as gdn
        if c["op"] == "prefill":
            return gdn.linear_prefill(c["q"], c["k"], c["v"], c["g"], c["state_in"], c["cu"])
        if c["op"] == "decode":
            return gdn.linear_decode(c["q"], c["k"], c["v"], c["g"], c["state"]), c["state"]
        if c["op"] == "park":
            gdn.state_store(c["state"], c["codes"], c["exps"], c["slot"])
        return gdn.state_load(c["codes"], c["exps"], c["slot"], state=c["out"])
    if c["op"] == "prefill":
        return _plain_prefill(c)
    if c["op"] == "decode":
        return _plain_decode(c)
    if c["op"] == "park":
        codes, exps = _quantise(c["state"], c["fmt"])
        c["codes"].view(torch.int8)[c["slot"].long()] = codes
        c["exps"][c["slot"].long()] = exps
    c["out"].copy_(_plain_load(c))
    return c["out"]


# -------------------------------------------------------------------- work ---
def work(case):
    c = case
    size = {"bf16": 2, "f16": 2, "f32": 4}
    rows = c["hv"] * c["dv"]
    if c["op"] == "prefill":
        T, io = sum(_lengths(c)), size[c["dtype"]]
        b = io * T * (2 * c["hqk"] * c["dk"] + 2 * rows) + 4 * c["hv"] * (1 if c["fixed"] else T)
        b += 4 * c["n"] * rows * c["dk"] * (2 if c["init"] else 1)
        return {"bytes": b, "flops": 4 * T * rows * c["dk"]}          # v k^T into the state, the state times q
    if c["op"] == "decode":
        io, s = size[c["dtype"]], size[c["sdtype"]]
        b = c["b"] * (io * (2 * c["hqk"] * c["dk"] + 2 * rows) + 2 * s * rows * c["dk"]) + 4 * c["hv"] * (1 if c["fixed"] else c["b"])
        return {"bytes": b, "flops": 5 * c["b"] * rows * c["dk"]}
    s = size[c["sdtype"]]
    values = c["n"] * rows * c["dk"]
    packed = values + values // min(32, c["dk"])
    # park: states in, codes and exponents out and in again, states out
    return {"bytes": values * s * (2 if c["op"] == "park" else 1) + packed * (2 if c["op"] == "park" else 1), "flops": 2 * values}


# ------------------------------------------------------------------- exact ---
def _two_to(e):
    """2.0 ** e for whole numbers in a tensor, from a table."""
    table = torch.tensor([math.ldexp(1.0, i) for i in range(-300, 301)], dtype=torch.float64, device=e.device)
    return table[e.long() + 300]


def exact(case, seed):
    """The definitions token by token, or value by value, in 64 bits."""
    c = prepare(case, seed)
    if c["op"] == "prefill":
        if max(c["lens"]) * c["n"] * c["hv"] > 8 * 8192 * 32 * 2:
            return None
        group, n = c["hv"] // c["hqk"], c["n"]
        head = torch.arange(c["hv"], device=DEV) // group
        S = torch.zeros(n, c["hv"], c["dv"], c["dk"], dtype=torch.float64, device=DEV) if c["state_in"] is None else c["state_in"].double()
        o = torch.empty(c["v"].shape, dtype=torch.float64, device=DEV)
        order = sorted(range(n), key=lambda i: -c["lens"][i])          # the longest first: those still running are a prefix
        start = [sum(c["lens"][:i]) for i in order]
        base, back = torch.tensor(start, device=DEV), torch.tensor(order, device=DEV)
        S = S[back]
        for t in range(max(c["lens"])):
            m = sum(x > t for x in c["lens"])
            i = base[:m] + t
            a = (c["g"].double() if c["g"].dim() == 1 else c["g"][i].double()).exp()
            k, v, q = c["k"][i][:, head].double(), c["v"][i].double(), c["q"][i][:, head].double()
            S[:m] = a[..., None, None] * S[:m] + v[..., None] * k[:, :, None, :]
            o[i] = torch.matmul(S[:m], q[..., None])[..., 0] / math.sqrt(c["dk"])
        out = torch.empty_like(S)
        out[back] = S
        return o, out
    if c["op"] == "decode":
        head = torch.arange(c["hv"], device=DEV) // (c["hv"] // c["hqk"])
        k, q, v = c["k"][:, head].double(), c["q"][:, head].double(), c["v"].double()
        S = torch.exp(c["g"].double())[..., None, None] * c["state"].double() + torch.einsum("bhi,bhj->bhij", v, k)
        return torch.einsum("bhij,bhj->bhi", S, q) / math.sqrt(c["dk"]), S
    if c["op"] == "load":
        slot = c["slot"].long()
        codes = c["codes"].view(torch.uint8)[slot].long()
        if c["fmt"] == "e4m3":
            sign, ex, man = codes >> 7, codes >> 3 & 15, codes & 7
            x = torch.where(ex == 0, man.double() / 512, (8 + man).double() * _two_to(ex - 10))
            x = torch.where(sign == 1, -x, x)
        else:
            x = torch.where(codes > 127, codes - 256, codes).double()
        return x * _two_to(c["exps"][slot].long() - 127).repeat_interleave(min(32, c["dk"]), -1)
    # park: quantised by the definition
    x = c["state"].double()
    big = x.abs().unflatten(-1, (-1, min(32, c["dk"]))).amax(-1).repeat_interleave(min(32, c["dk"]), -1)
    e = torch.floor(torch.log2(big.clamp_min(1e-60))) - 12
    for _ in range(15):                                                # the first power of two that is enough
        e = torch.where(big > QMAX[c["fmt"]] * _two_to(e), e + 1, e)
    e = e.clamp(-127, 127)
    y = x / _two_to(e)
    if c["fmt"] == "e4m3":                                             # 3 bits behind the leading one, steps of 2^-9 below 2^-6
        step = _two_to(torch.frexp(y.abs().clamp_min(2.0 ** -6))[1] - 4)
    else:
        step = torch.ones_like(y)
    return torch.round(y / step) * step * _two_to(e)
