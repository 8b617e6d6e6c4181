"""The quantised key/value cache's operators, as a user's program runs them, next to their plain forms.

Three operators, all on heads of 128 dims:

  write   new key and value rows quantised into the cache as they arrive, then read back as the values the cache
          now stands for;
  read    a stretch of the cache read back as bf16 keys and values;
  decode  attention of the newest queries over the quantised cache, with its log-sum-exp.

A cache row (one key or value head vector) is held in groups of `group` dims (32, 64 or 128). A group holds unsigned
codes n of `bits` bits (4 or 8), a bf16 scale s and a bf16 zero z, and stands for the values n * s + z, with

  z = min(x),  s = (max(x) - z) / (2^bits - 1) in fp32, rounded up to bf16,  n = round_half_even((x - z) / s).

Buffers: codes uint8 [B, H_kv, Tk, 128 * bits / 8] in dim order (4 bits: the even dim in the low half of its byte),
params bf16 [B, H_kv, Tk, 128 / group, 2] with (s, z) last. A sequence of length L (new tokens included) has its
i-th of T newest tokens at position L - T + i; positions below 0 are not there (not written, read as 0, and a
query there sees no key).
"""
import math
import random

import torch

own = False

D = 128


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # One new token for each of 64 sequences: what every layer does at every decode step. All latency.
        dict(name="write_step_d20", op="write", B=64, T=1, Hkv=10, Tk=2048, bits=4, group=64),
        # A training-sized batch of prompts written whole: bandwidth.
        dict(name="write_prompts_d20", op="write", B=32, T=2048, Hkv=10, Tk=2048, bits=4, group=32),
        # Left-padded prompts of mixed lengths into a longer 8-bit cache, odd sizes, one group a head.
        dict(name="write_ragged_8bit", op="write", B=7, T=1777, Hkv=13, Tk=2003, bits=8, group=128),
        # A few hundred rows of one sequence, as for a look at one prompt.
        dict(name="read_one_sequence", op="read", B=1, T=300, Hkv=5, Tk=4096, bits=8, group=64),
        # A whole 4-bit cache back in bf16, as before a pass that needs plain keys and values.
        dict(name="read_d20", op="read", B=32, T=2048, Hkv=10, Tk=2048, bits=4, group=64),
        # The smallest call: three short sequences, two new tokens, grouped heads. All latency.
        dict(name="decode_tiny", op="decode", B=3, H=4, Hkv=2, Tq=2, Tk=300, bits=4, group=32, min_len=1, window=-1),
        # Serving steps at d20 heads: 64 sequences with mixed lengths up to 2048.
        dict(name="decode_d20", op="decode", B=64, H=10, Hkv=10, Tq=1, Tk=2048, bits=4, group=64, min_len=1, window=-1),
        # The same with two query heads to a key/value head, in finer groups.
        dict(name="decode_d20_gqa", op="decode", B=64, H=10, Hkv=5, Tq=1, Tk=2048, bits=4, group=32, min_len=1,
             window=-1),
        # The same through a short-window layer, 8 bits.
        dict(name="decode_d20_sw_8bit", op="decode", B=64, H=10, Hkv=10, Tq=1, Tk=2048, bits=8, group=128, min_len=1,
             window=512),
        # Four long contexts, few rows: the work has to be split along the cache.
        dict(name="decode_long", op="decode", B=4, H=10, Hkv=5, Tq=1, Tk=65536, bits=4, group=64, min_len=50000,
             window=-1),
        # Eight new tokens at once over four query heads to a key/value head: the most rows a call takes.
        dict(name="decode_many_rows", op="decode", B=16, H=12, Hkv=3, Tq=8, Tk=4099, bits=4, group=128, min_len=100,
             window=-1),
        # A full serving batch: the largest call.
        dict(name="decode_d20_full", op="decode", B=256, H=10, Hkv=10, Tq=1, Tk=2048, bits=4, group=64, min_len=1024,
             window=-1),
    ]


_MOST_ROWS = 256 * 10 * 2048          # cache rows held (keys), at most
_MOST_BYTES = 540_000_000             # bytes of a pass, at most (below the largest listed case's)


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["write", "read", "decode", "decode"])
        c = dict(op=op, bits=rng.choice([4, 4, 8]), group=rng.choice([32, 64, 128]), Hkv=rng.randint(1, 13))
        c["B"] = _log_uniform(rng, 1, 256)
        if op == "decode":
            c["Tk"] = _log_uniform(rng, 1, 65536)
            G = rng.choice([1, 1, 1, 2, 2, 3, 4, 6, 8])
            c["H"] = G * c["Hkv"]
            c["Tq"] = min(rng.choice([1, 1, 1, 1, 2, 3, 4, 5, 8, 16]), 32 // G, c["Tk"])
            c["min_len"] = rng.choice([1, _log_uniform(rng, 1, c["Tk"])])
            c["window"] = _log_uniform(rng, 1, c["Tk"]) if rng.random() < 0.25 else -1
        else:
            c["Tk"] = _log_uniform(rng, 1, 8192)
            c["T"] = rng.choice([1, c["Tk"], _log_uniform(rng, 1, c["Tk"]), _log_uniform(rng, 1, c["Tk"])])
        if c["B"] * c["Hkv"] * c["Tk"] <= _MOST_ROWS and work(c)["bytes"] <= _MOST_BYTES:
            return c


def _lengths(case):
    """The sequences' lengths, the same set for every seed: evenly spread from the shortest to the capacity."""
    B, Tk = case["B"], case["Tk"]
    lo = case.get("min_len", 1)
    return [lo + int((Tk - lo) * (i + 1) / B) for i in range(B)] if B > 1 else [Tk]


def _row_bytes(case):
    return D * case["bits"] // 8 + 4 * (D // case["group"])


def work(case):
    lens, row, Hkv, B = _lengths(case), _row_bytes(case), case["Hkv"], case["B"]
    if case["op"] == "decode":
        H, Tq, w = case["H"], case["Tq"], case["window"]
        keys = sum(L if w < 0 else min(L, Tq + w) for L in lens)
        q_o = B * Tq * H * (2 * 2 * D + 4)
        seen = sum(min(p + 1, w + 1) if w >= 0 else p + 1 for L in lens for p in range(max(0, L - Tq), L))
        return {"bytes": keys * Hkv * 2 * row + q_o + 4 * B, "flops": 4 * D * H * seen}
    T = case["T"]
    rows = sum(min(L, T) for L in lens) * Hkv if op_aligned(case) else B * T * Hkv
    if case["op"] == "write":
        return {"bytes": rows * 2 * (2 * D + row) + B * T * Hkv * 2 * 2 * D + 4 * B, "flops": rows * 2 * D * 6}
    return {"bytes": rows * 2 * row + B * T * Hkv * 2 * 2 * D, "flops": rows * 2 * D * 2}


def op_aligned(case):
    """Whether the case's rows end at each sequence's length (written, or read by length) or start at 0."""
    return case["op"] == "write" or case["T"] < case["Tk"]


# ------------------------------------------------------------------------------------------------ plain forms

def _quantise(x, bits, group):
    """x fp32 [..., 128] (bf16 values) -> packed codes uint8 [..., 128 * bits / 8], params bf16 [..., 128/group, 2]."""
    levels = 2 ** bits - 1
    g = x.reshape(*x.shape[:-1], D // group, group)
    z = g.amin(-1, keepdim=True)
    span = g.amax(-1, keepdim=True) - z
    q = span / torch.full_like(span, float(levels))
    s = ((q.view(torch.int32) + 0xFFFF) & -65536).view(torch.float32)   # up to bf16 (the quotient is >= 0)
    n = torch.round((g - z) / torch.where(s > 0, s, torch.ones_like(s))).clamp(0, levels)
    codes = n.reshape(x.shape).to(torch.uint8)
    if bits == 4:
        codes = codes[..., 0::2] | (codes[..., 1::2] << 4)
    return codes, torch.cat([s, z], -1).to(torch.bfloat16)


def _values(codes, params, bits, group):
    """The fp32 values [..., 128] that codes and params stand for."""
    if bits == 4:
        codes = torch.stack([codes & 15, codes >> 4], -1)
    p = params.float()
    n = codes.reshape(*params.shape[:-1], group).float()
    return (n * p[..., 0:1] + p[..., 1:2]).reshape(*params.shape[:-2], D)


def _positions(lens, T, Tk):
    """Position of each of the T newest tokens, [B, T]; below 0 where it is not there."""
    return lens.clamp(0, Tk).long()[:, None] - T + torch.arange(T, device=lens.device)[None, :]


def _rows(cache, at):
    """The four buffers' rows at positions `at` [B, T], head by head: [B, T, H_kv, ...]."""
    b = torch.arange(at.shape[0], device=at.device)[:, None]
    return [t[b, :, at] for t in cache]


def _plain_write(s):
    T, Tk = s["k"].shape[1], s["cache"][0].shape[2]
    at = _positions(s["lens"], T, Tk)
    # a token below position 0 stands in for the one at position 0, whose row it then writes once more
    src = torch.arange(T, device=at.device)[None, :] - at.clamp(max=0)
    to = at.clamp(min=0)
    b = torch.arange(at.shape[0], device=at.device)[:, None]
    new = [*_quantise(s["k"].float()[b, src], s["bits"], s["group"]), *_quantise(s["v"].float()[b, src], s["bits"], s["group"])]
    kc, kp, vc, vp = s["cache"]
    kc[b, :, to], kp[b, :, to], vc[b, :, to], vp[b, :, to] = new
    return _plain_read(s)


def _plain_read(s):
    if s["lens"] is None:
        kc, kp, vc, vp = (t[:, :, :s["T"]].transpose(1, 2) for t in s["cache"])
        return {"k": _values(kc, kp, s["bits"], s["group"]).to(torch.bfloat16),
                "v": _values(vc, vp, s["bits"], s["group"]).to(torch.bfloat16)}
    at = _positions(s["lens"], s["T"], s["cache"][0].shape[2])
    kc, kp, vc, vp = _rows(s["cache"], at.clamp(min=0))
    there = (at >= 0)[:, :, None, None]
    k, v = _values(kc, kp, s["bits"], s["group"]), _values(vc, vp, s["bits"], s["group"])
    return {"k": torch.where(there, k, torch.zeros_like(k)).to(torch.bfloat16),
            "v": torch.where(there, v, torch.zeros_like(v)).to(torch.bfloat16)}


def _plain_decode(s):
    kc, kp, vc, vp = s["cache"]
    q = s["q"].float()
    B, Tq, H, _ = q.shape
    Hkv, Tk = kc.shape[1], kc.shape[2]
    G = H // Hkv
    k, v = _values(kc, kp, s["bits"], s["group"]), _values(vc, vp, s["bits"], s["group"])
    at = _positions(s["lens"], Tq, Tk)                                              # [B, Tq]
    j = torch.arange(Tk, device=q.device)[None, None, :]
    sees = j <= at[:, :, None]
    if s["window"] >= 0:
        sees = sees & (j >= at[:, :, None] - s["window"])
    rows = q.reshape(B, Tq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Tq, D)
    x = (rows @ k.transpose(2, 3)) * s["scale"]
    sees = sees[:, None, None].expand(B, 1, G, Tq, Tk).reshape(B, 1, G * Tq, Tk)
    x = x.masked_fill(~sees, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m > -math.inf, m, torch.zeros_like(m)))
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (m + torch.log(total)).reshape(B, Hkv, G, Tq).reshape(B, H, Tq)
    o = o.reshape(B, Hkv, G, Tq, D).permute(0, 3, 1, 2, 4).reshape(B, Tq, H, D)
    return {"o": o.to(torch.bfloat16), "lse": lse}


# ------------------------------------------------------------------------------------------------ one pass

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    B, Hkv, Tk, bits, group = (case[n] for n in ("B", "Hkv", "Tk", "bits", "group"))

    def normed(*shape):  # heads as they leave the QK normalisation: rms 1
        x = torch.randn(shape, generator=g, device=dev)
        return x.mul_(torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def projected(*shape):  # values as a projection leaves them: rows of different norms
        x = torch.randn(shape, generator=g, device=dev)
        return x.mul_(torch.exp(0.5 * torch.randn((*shape[:-1], 1), generator=g, device=dev))).to(torch.bfloat16)

    order = torch.randperm(B, generator=g, device=dev)
    lens = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)[order]
    s = {"op": case["op"], "bits": bits, "group": group, "lens": lens}
    if case["op"] == "write":
        s["T"] = case["T"]
        s["k"], s["v"] = normed(B, case["T"], Hkv, D), projected(B, case["T"], Hkv, D)
        row, n = D * bits // 8, D // group
        s["cache"] = tuple(t for _ in range(2) for t in (
            torch.zeros((B, Hkv, Tk, row), dtype=torch.uint8, device=dev),
            torch.zeros((B, Hkv, Tk, n, 2), dtype=torch.bfloat16, device=dev)))
        return s
    s["cache"] = (*_quantise(normed(B, Hkv, Tk, D).float(), bits, group),
                  *_quantise(projected(B, Hkv, Tk, D).float(), bits, group))
    if case["op"] == "read":
        s["T"] = case["T"]
        if not op_aligned(case):
            s["lens"] = None
        return s
    s["q"] = normed(B, case["Tq"], case["H"], D)
    s["scale"], s["window"] = 1.0 / math.sqrt(D), case["window"]
    return s


def run(state):
    s = state
    if own:
        import causal_self_attention_bf16_b200 as attn
        if s["op"] == "decode":
            o, lse = attn.attn_decode_kvq(s["q"], s["cache"], s["lens"], s["scale"],
                                          window=None if s["window"] < 0 else s["window"])
            return {"o": o, "lse": lse}
        if s["op"] == "write":
            attn.kvq_write(s["cache"], s["k"], s["v"], s["lens"])
        k, v = attn.kvq_read(s["cache"], s["T"], s["lens"])
        return {"k": k, "v": v}
    return {"write": _plain_write, "read": _plain_read, "decode": _plain_decode}[s["op"]](s)


# ------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """The definition in 64 bits, one sequence after another."""
    s = prepare(case, seed)
    bits, group, Tk, Hkv = case["bits"], case["group"], case["Tk"], case["Hkv"]
    lens = [Tk] * case["B"] if s["lens"] is None else s["lens"].tolist()
    top = float(2 ** bits - 1)

    def stands_for(codes, params):  # [..., bytes], [..., n, 2] -> fp64 [..., 128]
        c = codes.to(torch.int64)
        nib = [(c >> sh) & (15 if bits == 4 else 255) for sh in ((0, 4) if bits == 4 else (0,))]
        n = torch.stack(nib, -1).flatten(-2).double()
        sc = params[..., 0].double().repeat_interleave(group, -1)
        return n * sc + params[..., 1].double().repeat_interleave(group, -1)

    if case["op"] in ("write", "read"):
        T = case["T"]
        out = {}
        for name, at in (("k", 0), ("v", 2)):
            y = torch.zeros((case["B"], T, Hkv, D), dtype=torch.float64, device=s["cache"][0].device)
            for b, L in enumerate(lens):
                first = L - T if s["lens"] is not None else 0
                i0 = max(0, -first)
                if case["op"] == "read":
                    y[b, i0:] = stands_for(s["cache"][at][b, :, first + i0:first + T],
                                           s["cache"][at + 1][b, :, first + i0:first + T]).transpose(0, 1)
                    continue
                x = s[name][b, i0:].double().unflatten(-1, (D // group, group))
                low, high = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
                quotient = ((high - low).float() / torch.tensor([top], dtype=torch.float32, device=x.device)).double()
                # the least bf16 (8 significant bits) that is not below the quotient
                fraction, exponent = torch.frexp(quotient)
                step = torch.ldexp(torch.ceil(fraction * 256), exponent - 8)
                n = torch.where(step > 0, ((x - low) / step.clamp(min=1e-300)).round(), torch.zeros_like(x)).clamp(0, top)
                y[b, i0:] = (n * step + low).flatten(-2)
            out[name] = y
        return out

    B, Tq, H, _ = s["q"].shape
    if B * Hkv * Tk * 128 > 2 ** 31:
        return None
    o = torch.zeros((B, Tq, H, D), dtype=torch.float64, device=s["q"].device)
    lse = torch.full((B, H, Tq), -math.inf, dtype=torch.float64, device=s["q"].device)
    for b, L in enumerate(lens):
        k = stands_for(s["cache"][0][b, :, :L], s["cache"][1][b, :, :L]).repeat_interleave(H // Hkv, 0)
        v = stands_for(s["cache"][2][b, :, :L], s["cache"][3][b, :, :L]).repeat_interleave(H // Hkv, 0)
        for i in range(Tq):
            last = L - Tq + i
            if last < 0:
                continue
            first = 0 if case["window"] < 0 else max(0, last - case["window"])
            x = torch.einsum("hd,hjd->hj", s["q"][b, i].double(), k[:, first:last + 1]) * s["scale"]
            lse[b, :, i] = torch.logsumexp(x, -1)
            o[b, i] = torch.einsum("hj,hjd->hd", torch.softmax(x, -1), v[:, first:last + 1])
    return {"o": o, "lse": lse}


if __name__ == "__main__":
    for c in listed():
        w = work(c)
        print("%-22s %10.3f MB %10.3f GFLOP" % (c["name"], w["bytes"] / 1e6, w["flops"] / 1e9))
    r = random.Random(0)
    for _ in range(8):
        c = draw(r)
        print(c, "%.3f MB" % (work(c)["bytes"] / 1e6))
