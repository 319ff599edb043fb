"""Measured cases of the attention operators over the paged 8-bit key/value cache.

Three operators, each in its plain form (elementary torch operations in 32 bits) and, with ``own`` set, as the
package's entry points ``attn_append``, ``attn_decode`` and ``attn_prefill``.

The cache: e4m3 codes ``[n_pages][n_kv_heads][page][128]`` for keys and for values, a power-of-two float32 scale
for each page and head, and an int32 page table per sequence. A code is itself a floating value, returned as
``float8_e4m3fn`` beside its scale; the held value is their product.

A call's tokens are rows ``q_start[b] .. q_start[b+1]`` of sequence b; with ``n`` of them and ``kv_len[b]`` tokens in the
sequence's cache after the call's own, token i is at position ``kv_len[b] - n + i`` (below zero: a padding row).
"""
import math

import torch

own = False

D = 128           # head dimension
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -100


# ---------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one user typing: one token of one sequence is rotated and appended
        _case("append_1x1", "append", B=1, n=1, L=1000, Hq=16, Hkv=2, P=64),
        # a decode batch of 64 sequences of different lengths, one token each
        _case("append_64x1", "append", B=64, n=1, L=8191, spread=0.9, Hq=32, Hkv=8, P=64),
        # a prompt batch: 4 sequences of 8192 tokens, rows of a fused q|k|v projection
        _case("append_4x8192", "append", B=4, n=8192, L=8192, Hq=16, Hkv=4, P=64, fused=True),
        # prompt chunks of odd lengths in float32 behind earlier tokens, pairs interleaved, part of the head rotated
        _case("append_f32_ragged", "append", B=5, n=777, L=2049, spread=0.5, nspread=0.8, Hq=6, Hkv=2, P=16,
              dtype="f32", rot=64, interleaved=True),
        # one user, a short context: latency counts
        _case("decode_1x1000", "decode", B=1, n=1, L=1000, Hq=16, Hkv=2, P=64),
        # a full serving batch, contexts between 800 and 8191 tokens, with padding slots of a fixed-size batch
        _case("decode_64_ragged", "decode", B=64, n=1, L=8191, spread=0.9, Hq=32, Hkv=8, P=64, pad=3),
        # one user with a very long context
        _case("decode_1x131071", "decode", B=1, n=1, L=131071, Hq=32, Hkv=4, P=128),
        # drafts of 4 tokens of 32 sequences checked in one call, scores capped
        _case("verify_32x4", "decode", B=32, n=4, L=4100, spread=0.5, Hq=32, Hkv=4, P=32, softcap=30.0),
        # two short prompts
        _case("prefill_2x200", "prefill", B=2, n=200, L=200, nspread=0.4, Hq=16, Hkv=2, P=64),
        # a prompt batch: 4 sequences of 8192 tokens
        _case("prefill_4x8192", "prefill", B=4, n=8192, L=8192, Hq=16, Hkv=4, P=64),
        # the next chunk of 1024 tokens behind a context of 32768
        _case("prefill_chunk_33792", "prefill", B=1, n=1024, L=33792, Hq=32, Hkv=4, P=128, softcap=50.0),
        # prompts of odd lengths in a layer with a sliding window
        _case("prefill_window", "prefill", B=6, n=3001, L=4500, spread=0.3, nspread=0.6, Hq=6, Hkv=2, P=16,
              window=1000),
    ]


def _case(name, op, *, B, n, L, Hq, Hkv, P, spread=0.0, nspread=0.0, pad=0, dtype="bf16", rot=D, interleaved=False,
          fused=False, softcap=0.0, window=0):
    c = {"op": op, "B": B, "n": n, "L": L, "Hq": Hq, "Hkv": Hkv, "P": P, "spread": spread, "nspread": nspread, "pad": pad}
    if op == "append":
        c.update(dtype=dtype, rot=rot, interleaved=interleaved, fused=fused)
    else:
        c.update(softcap=softcap, window=window)
    return {"name": name, **c} if name else c


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = min(hi, max(lo, v))
    return v + 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(["append", "decode", "prefill"])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8] if Hkv < 8 else [1, 2, 4])
    P = rng.choice([16, 32, 64, 128])
    spread, Hq = rng.choice([0.0, 0.3, 0.9]), G * Hkv
    if op == "append":
        n, dtype = rng.choice([1, 1, _log_int(rng, 2, 8192)]), rng.choice(["bf16", "bf16", "f32"])
        B = _log_int(rng, 1, max(1, min(64, (24576 if dtype == "bf16" else 12288) // n)))
        L = n + _log_int(rng, 1, 4096)
        return _case("", op, B=B, n=n, L=L, Hq=min(Hq, 16) if n > 64 else Hq, Hkv=Hkv if Hq <= 16 or n <= 64 else 4, P=P,
                     spread=spread, nspread=rng.choice([0.0, 0.7]), dtype=dtype,
                     rot=rng.choice([32, 64, 128, 128]), interleaved=rng.random() < 0.3, fused=rng.random() < 0.5)
    window = rng.choice([0, 0, 0, _log_int(rng, 5, 4000)])
    softcap = rng.choice([0.0, 0.0, 30.0])
    if op == "decode":
        n = rng.choice([1, 1, 1, 2, 4, 8])
        L = n + _log_int(rng, 1, 131000)
        B = _log_int(rng, 1, max(1, min(64, 64 * 8 * 4096 // (L * Hkv))))
        return _case("", op, B=B, n=n, L=L, Hq=Hq, Hkv=Hkv, P=P, spread=spread, pad=min(B - 1, rng.choice([0, 0, 2])),
                     window=window, softcap=softcap)
    n = _log_int(rng, 9, 8192)
    L = max(n, min(n + rng.choice([0, _log_int(rng, 1, 24000)]), int(2e9 / (n * Hq))))
    L += L == 3072
    B = _log_int(rng, 1, max(1, min(8, int(2e9 / (n * L * Hq)))))
    return _case("", op, B=B, n=n, L=L, Hq=Hq, Hkv=Hkv, P=P, spread=spread, nspread=rng.choice([0.0, 0.6]), window=window,
                 softcap=softcap)


def _lengths(c):
    """(tokens in the call, tokens in the cache after it) of each sequence."""
    B, ns, Ls = c["B"], [], []
    for b in range(B):
        part = ((b * 37 + 11) % B) / B
        n = max(1, int(c["n"] * (1 - c["nspread"] * part)))
        L = max(n, int(c["L"] * (1 - c["spread"] * part)))
        ns.append(n)
        Ls.append(0 if b >= B - c["pad"] else L)
    return ns, Ls


def _visible(c, n, L):
    """(keys that each of the n tokens sees, first key that any sees)."""
    lo = [max(0, L - n + i + 1 - c["window"]) if c["window"] else 0 for i in range(n)]
    return [max(0, L - n + i + 1 - lo[i]) for i in range(n)], min(lo)


def work(c):
    ns, Ls = _lengths(c)
    N, Hq, Hkv, P = sum(ns), c["Hq"], c["Hkv"], c["P"]
    if c["op"] == "append":
        es = 2 if c["dtype"] == "bf16" else 4
        blocks = sum(-(-L // P) - (L - n) // P for n, L in zip(ns, Ls) if L)
        return {"bytes": N * D * (Hq * (es + 2) + 2 * Hkv * (es + 1)) + N * c["rot"] * 4 + blocks * Hkv * 16,
                "flops": N * c["rot"] * 3 * (Hq + Hkv) + 2 * N * Hkv * D}
    pairs = keys = 0
    for n, L in zip(ns, Ls):
        if L:
            seen, lo = _visible(c, n, L)
            pairs += sum(seen)
            keys += L - lo
    return {"bytes": keys * Hkv * 2 * (D + 4 / P) + N * Hq * D * 4, "flops": pairs * Hq * 4 * D}


# ---------------------------------------------------------------------------------------------------- inputs
def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s, at least 2^-100."""
    m, e = torch.frexp(amax)
    return torch.ldexp(torch.ones_like(amax), e - 9 + (m > 0.875).to(e.dtype)).clamp_min(MIN_SCALE)


def _pages(gen, n_pages, Hkv, P, dev):
    """Codes and scales of pages of normal values, a few channels of each head four times as large."""
    x = torch.randn(n_pages, Hkv, P, D, generator=gen, device=dev)
    x *= 1 + 3 * (torch.rand(1, Hkv, 1, D, generator=gen, device=dev) < 0.03).float()
    s = _pow2_scale(x.abs().amax((2, 3)))
    return (x / s[:, :, None, None]).to(torch.float8_e4m3fn), s


def prepare(c, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    ns, Ls = _lengths(c)
    B, Hq, Hkv, P, N = c["B"], c["Hq"], c["Hkv"], c["P"], sum(ns)
    width = -(-max(c["L"], 1) // P)
    used = [-(-L // P) for L in Ls]
    n_pages = sum(used) + 2
    order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros(B, width, dtype=torch.int32, device=dev)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    st = {"case": c, "N": N, "table": table,
          "q_start": torch.tensor([0] + ns, device=dev).cumsum(0).to(torch.int32),
          "kv_len": torch.tensor(Ls, dtype=torch.int32, device=dev)}
    st["k"], st["ks"] = _pages(gen, n_pages, Hkv, P, dev)
    st["v"], st["vs"] = _pages(gen, n_pages, Hkv, P, dev)
    if c["op"] == "append":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        widths = [Hq * D, Hkv * D, Hkv * D]
        if c["fused"]:
            row = torch.randn(N, sum(widths), generator=gen, device=dev).to(dt)
            parts = row.split(widths, 1)
        else:
            parts = [torch.randn(N, w, generator=gen, device=dev).to(dt) for w in widths]
        st["q_in"], st["k_in"], st["v_in"] = (p.unflatten(1, (-1, D)) for p in parts)
        pos = torch.arange(max(c["L"], 1), dtype=torch.float64, device=dev)[:, None]
        freq = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev) / c["rot"])
        st["cos"], st["sin"] = (pos * freq).cos().float(), (pos * freq).sin().float()
        st["q"] = torch.empty(N, Hq, D, dtype=torch.bfloat16, device=dev)
    else:
        st["q"] = (2 * torch.randn(N, Hq, D, generator=gen, device=dev)).to(torch.bfloat16)
        st["out"] = torch.empty_like(st["q"])
    # which sequence each token belongs to, for the plain form's gathers
    st["seq"] = torch.repeat_interleave(torch.arange(B, device=dev), torch.tensor(ns, device=dev))
    if own:
        _plan(st)
    return st


def _plan(st):
    """The handles that a serving program keeps: the cache, the dimensions, the rotation table and a workspace."""
    import gated_delta_ssm_gb300 as gdn
    c = st["case"]
    st["dims"] = gdn.AttnDims(n_seq=c["B"], n_q_heads=c["Hq"], n_kv_heads=c["Hkv"], page_size=c["P"],
                              n_pages=st["k"].shape[0], max_pages=st["table"].shape[1], n_tokens=st["N"], max_q=c["n"])
    st["cache"] = gdn.KvCache(st["k"], st["v"], st["ks"], st["vs"], st["table"])
    if c["op"] == "append":
        st["rope"] = gdn.Rope(st["cos"], st["sin"], interleaved=c["interleaved"])
    else:
        st["ws"] = torch.empty(gdn.attn_workspace_bytes(st["dims"], prefill=c["op"] == "prefill"), dtype=torch.uint8,
                               device="cuda")


# ---------------------------------------------------------------------------------------------------- one pass
def run(st):
    c = st["case"]
    if own:
        return _run_own(st, c)
    return _append(st, c) if c["op"] == "append" else _attend(st, c)


def _run_own(st, c):
    import gated_delta_ssm_gb300 as gdn
    if c["op"] == "append":
        gdn.attn_append(st["q_in"], st["k_in"], st["v_in"], st["cache"], st["q_start"], st["kv_len"], st["rope"], st["q"],
                        st["dims"])
        return {"q": st["q"], "k": st["k"], "v": st["v"], "ks": st["ks"], "vs": st["vs"]}
    call = gdn.attn_decode if c["op"] == "decode" else gdn.attn_prefill
    call(st["q"], st["cache"], st["q_start"], st["kv_len"], st["out"], st["dims"], scale=D ** -0.5, softcap=c["softcap"],
         window=c["window"], workspace=st["ws"])
    return st["out"]


def _positions(st):
    start, ln = st["q_start"].long(), st["kv_len"].long()
    i = torch.arange(st["N"], device=start.device) - start[st["seq"]]
    return i, ln[st["seq"]] - (start[1:] - start[:-1])[st["seq"]] + i


def _rotate(x, cos, sin, rot, interleaved):
    x = x.float()
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _append(st, c):
    P = c["P"]
    _, pos = _positions(st)
    rot = (st["cos"][pos], st["sin"][pos], c["rot"], c["interleaved"])
    st["q"].copy_(_rotate(st["q_in"], *rot))
    # the blocks that the call touches: [B][most blocks of a sequence], the last one again where there are fewer
    start, ln = st["q_start"].long(), st["kv_len"].long()
    n = start[1:] - start[:-1]
    first, last = (ln - n) // P, (ln - 1) // P
    most = (c["n"] + 2 * P - 2) // P
    blocks = torch.minimum(first[:, None] + torch.arange(most, device=first.device), last[:, None])
    touched = st["table"].gather(1, blocks).long().flatten()
    page, slot = st["table"][st["seq"], pos // P].long(), pos % P
    fresh = (blocks * P >= (ln - n)[:, None]).flatten()[:, None]
    for codes, scales, x in ((st["k"], st["ks"], _rotate(st["k_in"], *rot)), (st["v"], st["vs"], st["v_in"].float())):
        amax = torch.zeros_like(scales)
        amax.scatter_reduce_(0, page[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
        new = _pow2_scale(amax[touched])
        old = torch.where(fresh, new, scales[touched])
        new = torch.maximum(old, new)
        held = codes[touched].float() * (old / new)[:, :, None, None]
        codes[touched] = held.to(torch.float8_e4m3fn)
        scales[touched] = new
        codes[page, :, slot] = (x / scales[page][:, :, None]).to(torch.float8_e4m3fn)
    return {"q": st["q"], "k": st["k"], "v": st["v"], "ks": st["ks"], "vs": st["vs"]}


def _attend(st, c):
    B, n, Hkv, P = c["B"], c["n"], c["Hkv"], c["P"]
    G, L = c["Hq"] // Hkv, st["table"].shape[1] * P
    table, start, ln = st["table"].long(), st["q_start"].long(), st["kv_len"].long()
    j = torch.arange(L, device=table.device)
    held = (j < ln[:, None])[:, None, :, None]

    def gathered(codes, scales):
        x = codes[table].float() * scales[table][:, :, :, None, None]
        return torch.where(held, x.transpose(1, 2).reshape(B, Hkv, L, D), 0.0)

    count = start[1:] - start[:-1]
    i = torch.arange(n, device=table.device)
    rows = torch.minimum(start[:-1, None] + i, start[1:, None] - 1)
    pos = (ln - count)[:, None] + i
    q = st["q"][rows].float().reshape(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    s = torch.matmul(q, gathered(st["k"], st["ks"]).transpose(-1, -2)) * D ** -0.5
    if c["softcap"]:
        s = torch.tanh(s / c["softcap"]) * c["softcap"]
    seen = (j <= pos[:, :, None]) & (j < ln[:, None, None])
    if c["window"]:
        seen &= j > pos[:, :, None] - c["window"]
    s = s.view(B, Hkv, G, n, L).masked_fill_(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, G * n, L), gathered(st["v"], st["vs"])).view(B, Hkv, G, n, D)
    o = o / torch.where(total == 0, 1.0, total)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, c["Hq"], D)
    at, _ = _positions(st)
    st["out"].copy_(o[st["seq"], at])
    return st["out"]


# ---------------------------------------------------------------------------------------------------- in 64 bits
def exact(c, seed):
    """The operators' definitions in 64 bits, one sequence and head at a time."""
    st = prepare(c, seed)
    ns, Ls = _lengths(c)
    Hq, Hkv, P = c["Hq"], c["Hkv"], c["P"]
    table = st["table"].tolist() if c["op"] == "append" else st["table"].long()
    if c["op"] == "append":
        return _exact_append(st, c, ns, Ls, table)
    G, row = Hq // Hkv, 0
    out = torch.zeros(st["N"], Hq, D, dtype=torch.float64, device="cuda")
    for b, (n, L) in enumerate(zip(ns, Ls)):
        for h in range(Hkv if L else 0):
            pages = table[b, :-(-L // P)]
            k = (st["k"][pages, h].double() * st["ks"][pages, h].double()[:, None, None]).reshape(-1, D)[:L]
            v = (st["v"][pages, h].double() * st["vs"][pages, h].double()[:, None, None]).reshape(-1, D)[:L]
            for i0 in range(0, n, 2048):
                i1 = min(n, i0 + 2048)
                pos = torch.arange(L - n + i0, L - n + i1, device="cuda")
                lo = max(0, L - n + i0 + 1 - c["window"]) if c["window"] else 0
                hi = L - n + i1
                q = st["q"][row + i0:row + i1, h * G:(h + 1) * G].double()
                s = torch.einsum("igd,jd->gij", q, k[lo:hi]) / math.sqrt(D)
                if c["softcap"]:
                    s = c["softcap"] * torch.tanh(s / c["softcap"])
                j = torch.arange(lo, hi, device="cuda")
                hide = j[None] > pos[:, None]
                if c["window"]:
                    hide |= j[None] <= pos[:, None] - c["window"]
                s.masked_fill_(hide, -math.inf)
                w = torch.softmax(s, -1)
                out[row + i0:row + i1, h * G:(h + 1) * G] = torch.einsum("gij,jd->igd", w, v[lo:hi])
        row += n
    return out


def _exact_append(st, c, ns, Ls, table):
    P, rot = c["P"], c["rot"]
    half = rot // 2
    lead = torch.arange(half, device="cuda")
    ia, ib = (2 * lead, 2 * lead + 1) if c["interleaved"] else (lead, lead + half)
    pos = torch.cat([torch.arange(L - n, L, device="cuda") for n, L in zip(ns, Ls)])
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), torch.zeros((), dtype=torch.float64, device="cuda"))
    turn = turn * torch.complex(st["cos"][pos].double(), st["sin"][pos].double())[:, None]

    def rotated(x):
        y = x.double().clone()
        z = torch.complex(y[..., ia], y[..., ib]) * turn
        y[..., ia], y[..., ib] = z.real, z.imag
        return y

    codes = {"k": st["k"].clone(), "v": st["v"].clone()}
    scales = {"k": st["ks"].clone(), "v": st["vs"].clone()}
    for name, x in (("k", rotated(st["k_in"])), ("v", st["v_in"].double())):
        row = 0
        for b, (n, L) in enumerate(zip(ns, Ls)):
            # whole blocks at once where the call fills them, the ragged ends one by one
            for p0, p1 in _spans(L - n, L, P):
                count = -(-p1 // P) - p0 // P
                pages = torch.tensor(table[b][p0 // P:p0 // P + count], device="cuda")
                new = x[row + p0 - (L - n):row + p1 - (L - n)].unflatten(0, (count, -1)).transpose(1, 2)
                top = new.abs().amax((2, 3))
                s = torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX)).clamp_min(-100.0))
                s = torch.where(top > s * E4M3_MAX, 2 * s, torch.where(top <= s / 2 * E4M3_MAX, s / 2, s)).clamp_min(MIN_SCALE)
                if p0 % P:
                    old = scales[name][pages].double()
                    s = torch.maximum(s, old)
                    held = codes[name][pages].double() * (old / s)[:, :, None, None]
                    codes[name][pages] = held.float().to(torch.float8_e4m3fn)
                scales[name][pages] = s.float()
                unit = (new / s[:, :, None, None])
                at = p0 % P
                codes[name][pages, :, at:at + new.shape[2]] = _round_e4m3(unit)
            row += n
    return {"q": rotated(st["q_in"]), "k": codes["k"], "v": codes["v"], "ks": scales["k"].double(), "vs": scales["v"].double()}


def _spans(lo, hi, P):
    """[lo, hi) as a ragged head, whole blocks and a ragged tail."""
    cut0, cut1 = min(hi, -(-lo // P) * P), max(lo, hi // P * P)
    if cut0 >= cut1:
        spans = [(lo, cut0), (cut0, hi)]
    else:
        spans = [(lo, cut0), (cut0, cut1), (cut1, hi)]
    return [(a, b) for a, b in spans if a < b]


def _round_e4m3(x):
    """Round 64-bit values of at most 448 to e4m3: 3 bits behind the leading one, steps of 2^-9 at least, ties to even."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 4).clamp_min(-9).double())
    return (torch.round(x / step) * step).float().to(torch.float8_e4m3fn)
