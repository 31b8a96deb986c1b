"""The serving operators as they are measured: attention over packed prompts,
writing new keys and values into a paged cache, and attention of one new
token over that cache.

`run` computes each in its plain form (elementary torch operations in 32
bits, rounded once at the end) or, where `own` is true, calls the library.
`exact` gives the same outputs from the operators' definitions in 64 bits.

Lengths are texts ("4096,17,1") or come from a rule in the case itself
("lens" absent: `batch` lengths between `lo` and `hi`, drawn from `mix`, the
first one `hi`), so that the work of a case is known from the case alone.
"""
import math
import random

import torch

own = False

LOG2E = 1.4426950408889634
E4M3_MAX = 448.0
KEY_BLOCK = 64  # keys that share one power-of-2 scale of P in the FP8 modes


def listed():
    return [
        # --- packed prompts, causal
        # three short requests that arrive together (256 tokens in all): latency
        dict(name="varlen_tiny_bf16", op="varlen", type="bf16", hq=2, hkv=2, dqk=128, lens_q="100,1,155", lens_k="100,1,155", causal=True),
        # a prefill batch of chat prompts, 4:1 grouped heads, one token to 4K
        dict(name="varlen_gqa_bf16", op="varlen", type="bf16", hq=32, hkv=8, dqk=128, causal=True,
             lens_q="4096,2048,1531,977,512,301,129,64,2900,1024,17,1", lens_k="4096,2048,1531,977,512,301,129,64,2900,1024,17,1"),
        # one document of 16K tokens packed with two shorter prompts
        dict(name="varlen_long_bf16", op="varlen", type="bf16", hq=32, hkv=8, dqk=128, causal=True, lens_q="16384,4000,777", lens_k="16384,4000,777"),
        # the multi-head latent shape (192 wide queries and keys), every head its own keys
        dict(name="varlen_mla_bf16", op="varlen", type="bf16", hq=16, hkv=16, dqk=192, causal=True, lens_q="8192,2500,1111,333", lens_k="8192,2500,1111,333"),
        # prompts processed in chunks: new tokens behind a prefix already seen, FP8 with Lean P
        dict(name="varlen_chunk_fp8", op="varlen", type="leanp", hq=32, hkv=8, dqk=128, causal=True, lens_q="2048,1000,512,1500", lens_k="8192,1000,4600,6001"),
        # --- one new token over the paged cache
        # a single chat just after its prompt: latency of the smallest step
        dict(name="decode_single_bf16", op="decode", type="bf16", hq=32, hkv=8, dqk=128, batch=1, lo=200, hi=200, mix=1, page=16),
        # a serving batch of 64 chats, up to 4K tokens each
        dict(name="decode_batch_bf16", op="decode", type="bf16", hq=32, hkv=8, dqk=128, batch=64, lo=1, hi=4096, mix=2, page=64),
        # two long documents: few rows, the cache's length has to be split
        dict(name="decode_long_bf16", op="decode", type="bf16", hq=32, hkv=8, dqk=128, batch=2, lo=16001, hi=32768, mix=3, page=64),
        # a large batch over an FP8 cache with a scale for each head, up to 16K tokens
        dict(name="decode_batch_fp8", op="decode", type="e4m3", hq=32, hkv=8, dqk=128, batch=128, lo=256, hi=16384, mix=4, page=128),
        # 192 wide keys, every head its own: no sharing between query heads
        dict(name="decode_mla_bf16", op="decode", type="bf16", hq=16, hkv=16, dqk=192, batch=16, lo=100, hi=8192, mix=5, page=32),
        # --- new keys and values into the cache
        # the step of 64 chats: one token each
        dict(name="append_step_bf16", op="append", type="bf16", hkv=8, dqk=128, batch=64, lo=1, hi=4095, mix=6, page=64, new=",".join(["1"] * 64)),
        # the prompts of a prefill batch, rounded to FP8 on the way
        dict(name="append_prompts_fp8", op="append", type="e4m3", hkv=8, dqk=128, batch=8, lo=1, hi=300, mix=7, page=128, new="4096,8192,1531,977,512,301,129,1"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(32, 8), (32, 32), (8, 2), (4, 1), (16, 1), (40, 8), (2, 2)]


def draw(rng):
    op = rng.choice(["varlen", "varlen", "decode", "decode", "append"])
    mla = rng.random() < 0.2
    hq, hkv = (16, 16) if mla else rng.choice(HEADS)
    dqk = 192 if mla else 128
    if op == "varlen":
        left, lq, lk = 16384, [], []
        for _ in range(_log_int(rng, 1, 24)):
            n = _log_int(rng, 1, 8192)
            if n > left:
                break
            left -= n
            more = _log_int(rng, 1, 4096) if rng.random() < 0.25 else 0
            lq.append(n)
            lk.append(n + more)
        return dict(op="varlen", type=rng.choice(["bf16", "bf16", "exact", "leanp"]), hq=hq, hkv=hkv, dqk=dqk, causal=rng.random() < 0.85,
                    lens_q=",".join(map(str, lq)), lens_k=",".join(map(str, lk)))
    batch = _log_int(rng, 1, 128)
    typ = rng.choice(["bf16", "e4m3"])
    page = rng.choice([16, 32, 64, 128, 256])
    mix = rng.randrange(1 << 20)
    if op == "decode":
        # at most what the largest listed case holds: about 1.1 G of cached bytes
        row = hkv * (dqk + 128) * (2 if typ == "bf16" else 1)
        hi = _log_int(rng, 1, max(1, min(32768, (1 << 30) // (row * batch))))
        return dict(op="decode", type=typ, hq=hq, hkv=hkv, dqk=dqk, batch=batch, lo=max(1, hi // rng.choice([1, 2, 64])), hi=hi, mix=mix, page=page)
    most = max(1, 15000 // batch)
    new = [_log_int(rng, 1, most) for _ in range(batch)]
    return dict(op="append", type=typ, hkv=hkv, dqk=dqk, batch=batch, lo=1, hi=_log_int(rng, 1, 2000), mix=mix, page=page, new=",".join(map(str, new)))


# ------------------------------------------------------------------ lengths
def _ints(text):
    return [int(x) for x in text.split(",")]


def _lens(case):
    rng = random.Random(case["mix"])
    return [case["hi"]] + [_log_int(rng, case["lo"], case["hi"]) for _ in range(case["batch"] - 1)]


def _cu(lens, dev):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device=dev)


def _visible(sq, sk, causal):
    """Pairs (query, key) of one sequence that attend: key c to query i where c <= i + sk - sq."""
    if not causal:
        return sq * sk
    if sq <= sk:
        return sq * (sk - sq) + sq * (sq + 1) // 2
    return sk * (sk + 1) // 2


def work(case):
    d = case["dqk"] + 128
    if case["op"] == "varlen":
        lq, lk, es = _ints(case["lens_q"]), _ints(case["lens_k"]), 2 if case["type"] == "bf16" else 1
        pairs = sum(_visible(a, b, case["causal"]) for a, b in zip(lq, lk))
        read = sum(lq) * case["hq"] * case["dqk"] * es + sum(lk) * case["hkv"] * d * es
        return {"bytes": read + sum(lq) * case["hq"] * (128 * 2 + 4), "flops": 2.0 * case["hq"] * pairs * d}
    es = 2 if case["type"] == "bf16" else 1
    if case["op"] == "decode":
        n = sum(_lens(case))
        pages = sum(-(-x // case["page"]) for x in _lens(case))
        rows = case["batch"] * case["hq"]
        return {"bytes": n * case["hkv"] * d * es + rows * (case["dqk"] * 2 + 128 * 2 + 4) + 4 * pages, "flops": 2.0 * n * case["hq"] * d}
    t = sum(_ints(case["new"]))
    return {"bytes": t * case["hkv"] * d * (2 + es), "flops": float(t * case["hkv"] * d) if es == 1 else 0.0}


# ------------------------------------------------------------------- inputs
def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _heads(g, n, h, d):
    """Queries or keys: N(0, 1) with a lognormal(0, 0.5) scale for each channel of a head."""
    return _normal(g, n, h, d) * torch.exp(0.5 * _normal(g, h, d))


def _to_e4m3(x):
    """One scale for the tensor: (codes, descale)."""
    descale = (x.abs().amax() / E4M3_MAX).reshape(1)
    return (x / descale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), descale


def _paged(case, g, lens):
    """A cache with room for `lens` (pages in a random order) and its block table."""
    page, hkv, dqk = case["page"], case["hkv"], case["dqk"]
    need = [-(-n // page) for n in lens]
    total, width = sum(need), max(need)
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    k, v = _heads(g, total * page, hkv, dqk), _normal(g, total * page, hkv, 128)
    s = {"table": table, "k_descale": None, "v_descale": None}
    if case["type"] == "e4m3":
        for x, name in ((k, "k"), (v, "v")):
            ds = x.abs().amax(dim=2).amax(dim=0) / E4M3_MAX
            s[name + "_descale"] = ds.contiguous()
            s[name + "_cache"] = (x / ds[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(total, page, hkv, -1)
    else:
        s["k_cache"], s["v_cache"] = (x.to(torch.bfloat16).view(total, page, hkv, -1) for x in (k, v))
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    hkv, dqk = case["hkv"], case["dqk"]
    if case["op"] == "varlen":
        lq, lk = _ints(case["lens_q"]), _ints(case["lens_k"])
        s = {"case": case, "lens_q": lq, "lens_k": lk, "cu_q": _cu(lq, "cuda"), "cu_k": _cu(lk, "cuda")}
        q, k, v = _heads(g, sum(lq), case["hq"], dqk), _heads(g, sum(lk), hkv, dqk), _normal(g, sum(lk), hkv, 128)
        for name, x in (("q", q), ("k", k), ("v", v)):
            if case["type"] == "bf16":
                s[name], s[name + "_descale"] = x.to(torch.bfloat16), None
            else:
                s[name], s[name + "_descale"] = _to_e4m3(x)
        return s
    lens = _lens(case)
    if case["op"] == "decode":
        s = _paged(case, g, lens)
        s.update(case=case, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        s["q"] = _heads(g, case["batch"], case["hq"], dqk).to(torch.bfloat16)
        return s
    new = _ints(case["new"])
    s = _paged(case, g, [a + b for a, b in zip(lens, new)])
    s.update(case=case, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), cu=_cu(new, "cuda"), new=new)
    s["k"], s["v"] = _heads(g, sum(new), hkv, dqk).to(torch.bfloat16), _normal(g, sum(new), hkv, 128).to(torch.bfloat16)
    return s


# --------------------------------------------------------------- plain forms
def _weights(y, mode):
    """Unnormalised weights of scores y (log2 domain, -inf where masked) and the reference that they are relative to."""
    if mode == "bf16":
        ref = y.amax(dim=-1, keepdim=True)
        ref = torch.where(torch.isinf(ref), torch.zeros_like(ref), ref)
        return torch.exp2(y - ref), ref
    # FP8: P of a block of 64 keys is rounded to e4m3 relative to 2^e, e = ceil(block maximum) - 8
    n = y.shape[-1]
    y = torch.nn.functional.pad(y, (0, -n % KEY_BLOCK), value=-math.inf)
    y = y.view(*y.shape[:-1], -1, KEY_BLOCK)
    top = y.amax(dim=-1, keepdim=True)
    none = torch.isinf(top)
    e = torch.where(none, torch.zeros_like(top), torch.ceil(top) - 8.0)
    if mode == "exact":
        p = torch.exp2(y - e).to(torch.float8_e4m3fn).float()
    else:  # the e4m3 code itself is 8 (y - e) + 56
        p = (torch.round(8.0 * (y - e)) + 56.0).clamp(0.0, 126.0).to(torch.uint8).view(torch.float8_e4m3fn).float()
    ref = torch.where(none, torch.full_like(e, -math.inf), e).amax(dim=-2, keepdim=True)
    ref = torch.where(torch.isinf(ref), torch.zeros_like(ref), ref)
    w = p * torch.exp2(torch.where(none, torch.zeros_like(e), e - ref))
    return w.flatten(-2)[..., :n], ref.squeeze(-1)


def _plain_varlen(s):
    case = s["case"]
    hq, hkv, mode = case["hq"], case["hkv"], case["type"]
    tq = s["q"].shape[0]
    c = case["dqk"] ** -0.5 * LOG2E
    vd = 1.0
    if mode != "bf16":
        c, vd = c * s["q_descale"] * s["k_descale"], s["v_descale"]
    out = torch.zeros((tq, hq, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((hq, tq), -math.inf, dtype=torch.float32, device="cuda")
    q0 = k0 = 0
    for sq, sk in zip(s["lens_q"], s["lens_k"]):
        q = s["q"][q0:q0 + sq].float().view(sq, hkv, hq // hkv, -1).permute(1, 2, 0, 3)  # (Hkv, G, Sq, d)
        k, v = s["k"][k0:k0 + sk].float().permute(1, 2, 0), s["v"][k0:k0 + sk].float().permute(1, 0, 2)
        seen = torch.arange(sk, device="cuda")[None, :] <= torch.arange(sq, device="cuda")[:, None] + (sk - sq)
        for g in range(hkv):  # one kv head at a time: the scores of a long prompt are large
            y = torch.matmul(q[g], k[g]) * c
            if case["causal"]:
                y.masked_fill_(~seen, -math.inf)
            w, ref = _weights(y, mode)
            del y
            total = w.sum(dim=-1, keepdim=True)
            o = torch.matmul(w, v[g]) / torch.where(total > 0, total, torch.ones_like(total)) * vd
            heads = slice(g * (hq // hkv), (g + 1) * (hq // hkv))
            out[q0:q0 + sq, heads] = o.permute(1, 0, 2).to(torch.bfloat16)
            lse[heads, q0:q0 + sq] = ((ref + torch.log2(total)) / LOG2E).squeeze(-1)
        q0, k0 = q0 + sq, k0 + sk
    return out, lse


def _pages(s, name):
    """The cache of every sequence in order, (B, keys, Hkv, d) in 32 bits, with its scale."""
    c = s[name + "_cache"]
    bits = torch.uint8 if s["k_descale"] is not None else torch.int16
    x = c.view(bits)[s["table"].clamp(min=0).long()].view(c.dtype).flatten(1, 2).float()
    return x if s["k_descale"] is None else x * s[name + "_descale"][:, None]


def _plain_decode(s):
    case = s["case"]
    b, hkv, g = case["batch"], case["hkv"], case["hq"] // case["hkv"]
    q = s["q"].float().view(b, hkv, g, -1)
    k = _pages(s, "k")
    y = torch.matmul(q, k.permute(0, 2, 3, 1)) * (case["dqk"] ** -0.5 * LOG2E)
    there = torch.arange(k.shape[1], device="cuda")[None, :] < s["lens"][:, None]
    del k
    y.masked_fill_(~there[:, None, None, :], -math.inf)
    w, ref = _weights(y, "bf16")
    total = w.sum(dim=-1, keepdim=True)
    v = _pages(s, "v")
    v.masked_fill_(~there[:, :, None, None], 0.0)  # what lies behind a sequence's last key is not data
    o = torch.matmul(w, v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (ref + torch.log2(total)) / LOG2E
    return o.reshape(b, -1, 128).to(torch.bfloat16), lse.reshape(b, -1)


def _plain_append(s):
    page = s["case"]["page"]
    cu, n = s["cu"].long(), s["k"].shape[0]
    t = torch.arange(n, device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = s["lens"].long()[b] + t - cu[b]
    slot = s["table"].long()[b, pos // page] * page + pos % page
    for name in ("k", "v"):
        x, cache = s[name], s[name + "_cache"]
        if s["k_descale"] is not None:
            x = (x.float() * (1.0 / s[name + "_descale"])[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(cache.dtype)
            cache, x = cache.view(torch.uint8), x.view(torch.uint8)
        cache.flatten(0, 1)[slot] = x
    return s["k_cache"], s["v_cache"]


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import bf16_causal_prefill_02_b200 as zq

        if op == "varlen":
            mode = {"softmax_mode": zq.ZQ_SOFTMAX_EXACT if s["case"]["type"] == "exact" else zq.ZQ_SOFTMAX_LEANP}
            return zq.attn_varlen(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=s["case"]["causal"],
                                  q_descale=s["q_descale"], k_descale=s["k_descale"], v_descale=s["v_descale"], **mode)
        if op == "decode":
            return zq.attn_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], k_descale=s["k_descale"], v_descale=s["v_descale"])
        return zq.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"],
                            k_descale=s["k_descale"], v_descale=s["v_descale"])
    return {"varlen": _plain_varlen, "decode": _plain_decode, "append": _plain_append}[op](s)


# ------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"varlen": _exact_varlen, "decode": _exact_decode, "append": _exact_append}[case["op"]](case, s)


def _attend64(q, k, v, visible, mode, scale):
    """Rows of q (R, d) over keys (S, d): o = sum w v / sum w and ln of the sum of weights; `visible` (R, S) or None."""
    x = (q.double() @ k.double().t()) * scale
    if visible is not None:
        x = torch.where(visible, x, torch.full_like(x, -math.inf))
    if mode == "bf16":
        lse = torch.logsumexp(x, dim=-1)
        w = torch.exp(x - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None])
        return w @ v.double(), lse
    y = x / math.log(2.0)
    num = torch.zeros((q.shape[0], v.shape[1]), dtype=torch.float64, device=q.device)
    den = torch.zeros((q.shape[0],), dtype=torch.float64, device=q.device)
    base = torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=q.device)
    for at in range(0, y.shape[1], KEY_BLOCK):
        z = y[:, at:at + KEY_BLOCK]
        e = torch.ceil(z.amax(dim=-1)) - 8
        some = ~torch.isinf(e)
        u = z - torch.where(some, e, torch.zeros_like(e))[:, None]
        if mode == "exact":
            p = torch.exp2(u).to(torch.float8_e4m3fn).double()
        else:
            code = torch.clamp(torch.round(8 * u) + 56, 0, 126)
            octave, part = torch.div(code, 8, rounding_mode="floor"), torch.remainder(code, 8)
            p = torch.where(octave > 0, (1 + part / 8) * torch.exp2(octave - 7), part * 2.0 ** -9)
        nbase = torch.maximum(base, e)
        fall = torch.where(torch.isinf(base), torch.zeros_like(base), torch.exp2(base - nbase))
        rise = torch.where(some, torch.exp2(e - nbase), torch.zeros_like(e))
        num = num * fall[:, None] + (p * rise[:, None]) @ v[at:at + KEY_BLOCK].double()
        den = den * fall + p.sum(dim=-1) * rise
        base = nbase
    ok = den > 0
    return torch.where(ok[:, None], num / den[:, None], torch.zeros_like(num)), torch.where(ok, torch.log(den) + base * math.log(2.0), base)


def _exact_varlen(case, s):
    hq, group, mode = case["hq"], case["hq"] // case["hkv"], case["type"]
    out = torch.zeros((s["q"].shape[0], hq, 128), dtype=torch.float64, device="cuda")
    lse = torch.full((hq, s["q"].shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    scale, vd = case["dqk"] ** -0.5, 1.0
    if mode != "bf16":
        scale, vd = scale * float(s["q_descale"].double() * s["k_descale"].double()), float(s["v_descale"])
    q0 = k0 = 0
    for sq, sk in zip(s["lens_q"], s["lens_k"]):
        visible = None
        if case["causal"]:
            visible = torch.ones((sq, sk), dtype=torch.bool, device="cuda").tril(sk - sq).repeat(group, 1)
        for g in range(case["hkv"]):  # the query heads of a kv head are rows over the same keys
            heads = slice(g * group, (g + 1) * group)
            q = s["q"][q0:q0 + sq, heads].permute(1, 0, 2).flatten(0, 1)
            o, l = _attend64(q, s["k"][k0:k0 + sk, g], s["v"][k0:k0 + sk, g], visible, mode, scale)
            out[q0:q0 + sq, heads], lse[heads, q0:q0 + sq] = o.view(group, sq, 128).permute(1, 0, 2) * vd, l.view(group, sq)
        q0, k0 = q0 + sq, k0 + sk
    return out, lse


def _exact_decode(case, s):
    group, page = case["hq"] // case["hkv"], case["page"]
    out = torch.zeros((case["batch"], case["hq"], 128), dtype=torch.float64, device="cuda")
    lse = torch.zeros((case["batch"], case["hq"]), dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(case)):
        at = s["table"][b, :-(-n // page)].long()
        k, v = (s[x + "_cache"].view(torch.uint8)[at].view(s[x + "_cache"].dtype).flatten(0, 1)[:n].double() for x in ("k", "v"))
        if case["type"] == "e4m3":
            k, v = k * s["k_descale"].double()[:, None], v * s["v_descale"].double()[:, None]
        x = torch.einsum("gjd,ngd->gjn", s["q"][b].double().view(-1, group, case["dqk"]), k) * case["dqk"] ** -0.5
        lse[b] = torch.logsumexp(x, dim=-1).flatten()
        out[b] = torch.einsum("gjn,ngd->gjd", torch.softmax(x, dim=-1), v).flatten(0, 1)
    return out, lse


def _exact_append(case, s):
    """The cache after the call: bf16 values as they are; e4m3 the code nearest to the 32-bit product of a value and the scale's reciprocal."""
    got = []
    for x in ("k", "v"):
        cache = s[x + "_cache"].double().flatten(0, 1)
        new = s[x].double()
        if case["type"] == "e4m3":
            inv = (1.0 / s[x + "_descale"].double()).float().double()
            new = (new * inv[:, None]).float().clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).double()
        at = 0
        for b, (have, n) in enumerate(zip(_lens(case), s["new"])):
            pos = torch.arange(have, have + n, device="cuda")
            cache[s["table"][b, pos // case["page"]].long() * case["page"] + pos % case["page"]] = new[at:at + n]
            at += n
        got.append(cache.view(s[x + "_cache"].shape))
    return tuple(got)
