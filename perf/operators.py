"""What a serving program asks of the library's batched-serving operators, as cases that can be timed.

Three operators, each in its plain form (elementary torch operations in 32 or 64 bits) and as
the library's call:

- ``packed``: causal attention over packed prompts of different lengths (``tfm.packed_attention``);
- ``prefix``: attention of one or a few new tokens per sequence over a prefix shared by the
  whole batch and each sequence's own cache (``tfm.prefix_attention``);
- ``verify``: verification of drafted tokens from given random numbers (``tfm.verify_draft``).

A case fixes the sizes and the lengths of its sequences; the values come from the seed.
"""
import random

import torch

own = False


# ------------------------------------------------------------------ the cases
def _packed(name, lens_seed, n_seq, longest, H, Hkv, dh, window=0, dtype="bf16", tail=0, heads_first=False):
    return {"name": name, "op": "packed", "lens_seed": lens_seed, "n_seq": n_seq, "longest": longest, "H": H, "Hkv": Hkv,
            "dh": dh, "window": window, "dtype": dtype, "tail": tail, "heads_first": heads_first}


def _prefix(name, lens_seed, B, T, prefix, longest, H, Hkv, dh):
    return {"name": name, "op": "prefix", "lens_seed": lens_seed, "B": B, "T": T, "prefix": prefix, "longest": longest,
            "H": H, "Hkv": Hkv, "dh": dh}


def _verify(name, lens_seed, B, K, V, temperature):
    return {"name": name, "op": "verify", "lens_seed": lens_seed, "B": B, "K": K, "V": V, "temperature": temperature}


def listed():
    return [
        # A handful of one-line chat turns arriving together, GPT-2-small heads: the call's latency.
        _packed("prompts_short", 1, 6, 48, 12, 12, 64),
        # A batch of uneven documents at the GPT-2-small shape (12 heads of 64, up to 1024 tokens).
        _packed("prompts_gpt2s", 2, 24, 1024, 12, 12, 64, heads_first=True),
        # Prompts of the grouped-query model (16 heads on 4, d_head 128, up to 2048 tokens); q, k, v token-major, and the
        # last rows of the buffers belong to no sequence.
        _packed("prompts_gqa", 3, 12, 2048, 16, 4, 128, tail=37),
        # The long-context shape: one prompt of 8192 tokens with two shorter ones behind it.
        _packed("prompts_long", 13, 3, 8192, 16, 16, 64),
        # The small model (16 heads of 32) with a sliding window of 256.
        _packed("prompts_window", 5, 32, 1000, 16, 16, 32, window=256),
        # The fp32 character model (4 heads of 16), many short lines.
        _packed("prompts_fp32", 6, 64, 300, 4, 4, 16, dtype="fp32"),
        # Four chats under a short system prompt, one token each: the latency of a step.
        _prefix("step_few", 7, 4, 1, 511, 64, 12, 12, 64),
        # A served batch of the grouped-query model under a system prompt of 2048 tokens.
        _prefix("step_gqa", 8, 64, 1, 2048, 600, 16, 4, 128),
        # Five drafted tokens for each of 16 answers about one long document.
        _prefix("step_draft", 9, 16, 5, 8192, 1000, 16, 4, 128),
        # Many short answers (votes, samples) over one long prompt, 16 heads of 64.
        _prefix("step_wide", 10, 192, 1, 16384, 300, 16, 16, 64),
        # One chat, four drafted tokens, the 32000-token vocabulary.
        _verify("verify_one", 11, 1, 4, 32000, 1.0),
        # A served batch, five drafted tokens each, the 50257-token vocabulary.
        _verify("verify_batch", 12, 64, 5, 50257, 0.8),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("packed", "packed", "prefix", "prefix", "verify"))
    s = rng.randrange(1 << 20)
    if op == "packed":
        dtype = rng.choice(("bf16", "bf16", "bf16", "fp32"))
        if dtype == "fp32":
            H, Hkv = rng.choice(((4, 4), (4, 2), (6, 1)))
            c = _packed("", s, _log(rng, 1, 64), _log(rng, 3, 400), H, Hkv, rng.choice((16, 32, 64)), rng.choice((0, 0, 33)), dtype)
        else:
            H, Hkv, dh = rng.choice(((12, 12, 64), (16, 4, 128), (16, 16, 64), (16, 16, 32), (8, 1, 128), (12, 4, 64), (6, 2, 128)))
            n = _log(rng, 1, 40)
            c = _packed("", s, n, _log(rng, 5, min(8192, 16000 // n)), H, Hkv, dh, rng.choice((0, 0, 0, 100, 512)), dtype,
                        rng.choice((0, 0, 19)), rng.choice((False, True)))
    elif op == "prefix":
        H, Hkv, dh = rng.choice(((12, 12, 64), (16, 4, 128), (16, 16, 64), (16, 16, 32), (8, 1, 128), (12, 4, 64)))
        B = _log(rng, 1, 192)
        c = _prefix("", s, B, rng.choice((1, 1, 1, 2, 5, 8)), _log(rng, 7, 16384), _log(rng, 9, min(2000, 50000 // B)), H, Hkv, dh)
    else:
        c = _verify("", s, _log(rng, 1, 64), rng.randint(1, 7), rng.choice((23, 10000, 32000, 50257, _log(rng, 50, 50000))),
                    rng.choice((1.0, 1.0, 0.7, 1.3, 0.0)))
    del c["name"]
    return c


def _lens(case):
    """The lengths of the case's sequences: uneven, the longest always there; a prompt or a cache may be empty, a sequence's
    own cache holds its T new tokens at least, and a sequence has between none and K drafted tokens."""
    rng = random.Random(case["lens_seed"])
    if case["op"] == "packed":
        n, longest = case["n_seq"], case["longest"]
        lens = [longest] + [_log(rng, 1, longest) if rng.random() < 0.5 else rng.randint(0, longest) for _ in range(n - 1)]
    elif case["op"] == "prefix":
        n, longest = case["B"], max(case["longest"], case["T"])
        lens = [longest] + [rng.randint(case["T"], longest) for _ in range(n - 1)]
    else:
        lens = [case["K"]] + [case["K"] if rng.random() < 0.75 else rng.randint(0, case["K"]) for _ in range(case["B"] - 1)]
    rng.shuffle(lens)
    return lens


def _pairs(L, window):
    """Visible (query, key) pairs of a causal sequence of L tokens, with a window if it is not 0."""
    w = min(window, L) if window else L
    return w * (w + 1) // 2 + (L - w) * w


def work(case):
    lens = _lens(case)
    if case["op"] == "packed":
        es, T = (2 if case["dtype"] == "bf16" else 4), sum(lens)
        return {"bytes": es * T * case["dh"] * 2 * (case["H"] + case["Hkv"]) + 4 * (len(lens) + 1),
                "flops": 4 * case["dh"] * case["H"] * sum(_pairs(L, case["window"]) for L in lens)}
    if case["op"] == "prefix":
        B, T, P, H, Hkv, dh = (case[k] for k in ("B", "T", "prefix", "H", "Hkv", "dh"))
        pairs = sum(P * T + T * L - T * (T - 1) // 2 for L in lens)
        return {"bytes": 4 * Hkv * dh * (P + sum(lens)) + 4 * B * H * T * dh + 4 * B, "flops": 4 * dh * H * pairs}
    B, K, V = case["B"], case["K"], case["V"]
    n = sum(lens)
    if case["temperature"] == 0:
        return {"bytes": 4 * V * (n + B) + 12 * B * (K + 1), "flops": V * (n + B)}
    return {"bytes": 4 * V * (n + B + n + B) + 16 * B * (K + 1), "flops": 4 * V * (2 * n + B) + 6 * V * B}


# ------------------------------------------------------------------ the inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens = _lens(case)

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    s = {"case": case}
    if case["op"] == "packed":
        T, H, Hkv, dh = sum(lens) + case["tail"], case["H"], case["Hkv"], case["dh"]
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32

        def rows(heads, std):       # [T, heads, dh], stored head-major (as the QKV projection writes it) or token-major
            if case["heads_first"]:
                return normal(heads, T, dh, dtype=dtype, std=std).transpose(0, 1)
            return normal(T, heads, dh, dtype=dtype, std=std)

        s["q"], s["k"], s["v"] = rows(H, 1.5), rows(Hkv, 1.0), rows(Hkv, 1.0)
        s["o"] = torch.zeros(T, H, dh, dtype=dtype, device="cuda")
        ends = torch.tensor([0] + lens).cumsum(0)
        s["cu"] = ends.to(torch.int32).cuda()
    elif case["op"] == "prefix":
        B, T, P, H, Hkv, dh = (case[k] for k in ("B", "T", "prefix", "H", "Hkv", "dh"))
        room = max(lens) + 64       # the caches go on being filled
        s["q"] = normal(B, H, T, dh, std=1.5)
        s["kp"], s["vp"] = normal(Hkv, P, dh), normal(Hkv, P, dh)
        s["kc"], s["vc"] = normal(B, Hkv, room, dh), normal(B, Hkv, room, dh)
        s["lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
        s["o"] = torch.zeros(B, T, H * dh, dtype=torch.bfloat16, device="cuda")
    else:
        B, K, V = case["B"], case["K"], case["V"]
        ld = (V + 3) // 4 * 4
        # The drafter follows the target with some error; drafted tokens are drawn from it.
        s["target"] = normal(B * (K + 1), ld, dtype=torch.float32, std=2.5)
        rows = s["target"].view(B, K + 1, ld)[:, :K].reshape(B * K, ld)
        s["draft_logits"] = rows + normal(B * K, ld, dtype=torch.float32, std=0.5)
        s["noise"] = torch.empty(B, ld, device="cuda").exponential_(generator=g).clamp_(min=1e-30)
        race = torch.empty(B * K, V, device="cuda").exponential_(generator=g).clamp_(min=1e-30)
        temp = case["temperature"] or 0.2
        drafted = (s["draft_logits"][:, :V] / temp).softmax(1).div(race).argmax(1)
        s["draft"] = drafted.view(B, K).to(torch.int32)
        s["n_draft"] = torch.tensor(lens, dtype=torch.int32).cuda()
        s["u"] = torch.rand(B, K, generator=g, device="cuda")
        s["tokens"] = torch.full((B, K + 1), -1, dtype=torch.int32, device="cuda")
        s["n_accepted"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
_space = {}


def _workspace(nbytes):
    """The one workspace that a serving program keeps, grown when a call needs more."""
    if "ws" not in _space or _space["ws"].numel() < nbytes:
        _space["ws"] = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")
    return _space["ws"]


def run(state):
    return {"packed": _run_packed, "prefix": _run_prefix, "verify": _run_verify}[state["case"]["op"]](state)


def _run_packed(s):
    c = s["case"]
    q, k, v, o, cu = s["q"], s["k"], s["v"], s["o"], s["cu"]
    if own:
        from decoder_only_transformer_gb300 import tfm
        ws = _workspace(tfm.packed_attention_workspace_bytes(q.shape[0], c["n_seq"]))
        tfm.packed_attention(q, k, v, o, cu, ws, window=c["window"])
        return o
    # Every sequence padded to the longest one, all heads at once.
    T, H, dh = q.shape
    G, n, L = H // c["Hkv"], c["n_seq"], c["longest"]
    start, length = cu[:-1].long(), (cu[1:] - cu[:-1]).long()
    at = torch.arange(L, device=q.device)
    there = at[None, :] < length[:, None]                                # [n, L]
    idx = (start[:, None] + at[None, :]).clamp(max=T - 1)
    qp = q[idx].float().view(n, L, c["Hkv"], G, dh).permute(0, 2, 3, 1, 4)
    kp = k[idx].float().permute(0, 2, 1, 3)[:, :, None]                  # [n, Hkv, 1, L, dh]
    vp = v[idx].float().permute(0, 2, 1, 3)[:, :, None]
    scores = qp @ kp.transpose(-1, -2) * dh ** -0.5
    seen = at[None, :] <= at[:, None]
    if c["window"]:
        seen = seen & (at[None, :] > at[:, None] - c["window"])
    scores.masked_fill_(~seen, float("-inf"))
    scores -= scores.amax(-1, keepdim=True)
    scores.exp_()
    scores /= scores.sum(-1, keepdim=True)
    out = (scores @ vp).permute(0, 3, 1, 2, 4).reshape(n, L, H, dh)
    full = torch.zeros(T, H, dh, dtype=q.dtype, device=q.device)
    full[idx[there]] = out[there].to(q.dtype)
    return full


def _run_prefix(s):
    c = s["case"]
    q, kp, vp, kc, vc, o, lens = (s[k] for k in ("q", "kp", "vp", "kc", "vc", "o", "lens"))
    B, H, T, dh = q.shape
    Hkv = c["Hkv"]
    if own:
        from decoder_only_transformer_gb300 import tfm
        ws = _workspace(tfm.prefix_attention_workspace_bytes(B, H, Hkv, T, dh))
        tfm.prefix_attention(q, kp, vp, kc, vc, o, lens, ws)
        return o
    G, P, R = H // Hkv, kp.shape[1], kc.shape[2]
    qf = q.float().view(B, Hkv, G * T, dh) * dh ** -0.5
    shared = qf.transpose(0, 1).reshape(Hkv, B * G * T, dh) @ kp.float().transpose(1, 2)
    shared = shared.view(Hkv, B, G, T, P).transpose(0, 1)
    mine = (qf @ kc.float().transpose(2, 3)).view(B, Hkv, G, T, R)
    last = lens.long()[:, None] - T + 1 + torch.arange(T, device=q.device)            # [B, T]: own keys that row t sees
    seen = torch.arange(R, device=q.device) < last[:, :, None]
    mine = mine.masked_fill(~seen[:, None, None], float("-inf"))
    top = torch.maximum(shared.amax(-1), mine.amax(-1))[..., None]
    shared, mine = (shared - top).exp(), (mine - top).exp()
    total = shared.sum(-1, keepdim=True) + mine.sum(-1, keepdim=True)
    a = shared.transpose(0, 1).reshape(Hkv, B * G * T, P) @ vp.float()
    a = a.view(Hkv, B, G, T, dh).transpose(0, 1)
    b = (mine.reshape(B, Hkv, G * T, R) @ vc.float()).view(B, Hkv, G, T, dh)
    return ((a + b) / total).to(q.dtype).reshape(B, H, T, dh).transpose(1, 2).reshape(B, T, H * dh)


def _run_verify(s):
    c = s["case"]
    B, K, V, temp = c["B"], c["K"], c["V"], c["temperature"]
    target, dlogits, draft, n_draft, u, noise = (s[k] for k in ("target", "draft_logits", "draft", "n_draft", "u", "noise"))
    if own:
        from decoder_only_transformer_gb300 import tfm
        ws = _workspace(tfm.verify_draft_workspace_bytes(B, K, V))
        tfm.verify_draft(target, dlogits, draft, n_draft, u, noise, V, s["tokens"], s["n_accepted"], ws, temperature=temp)
        return s["tokens"], s["n_accepted"]
    z = target.view(B, K + 1, -1)[..., :V]
    ids = draft.long()
    row = torch.arange(K, device=z.device)
    inside = row[None, :] < n_draft[:, None]
    if temp == 0:
        best = z.argmax(-1)                                             # [B, K + 1]
        ok = (ids == best[:, :K]) & inside
        n = ok.long().cumprod(1).sum(1)
        new = best.gather(1, n[:, None])
    else:
        # In 64 bits: a token next to the border between two others must not change with the rounding.
        p = (z.double() / temp).softmax(-1)
        q = (dlogits.view(B, K, -1)[..., :V].double() / temp).softmax(-1)
        px = p[:, :K].gather(2, ids[..., None])[..., 0]
        qx = q.gather(2, ids[..., None])[..., 0]
        ok = (u.double() * qx < px) & inside
        n = ok.long().cumprod(1).sum(1)
        pick = n[:, None, None].expand(B, 1, V)
        pn = p.gather(1, pick)[:, 0]
        qn = torch.cat([q, torch.zeros_like(q[:, :1])], 1).gather(1, pick)[:, 0]
        qn = torch.where((n < n_draft)[:, None], qn, torch.zeros_like(qn))
        rest = (pn - qn).clamp(min=0)
        rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, pn)
        new = (rest / noise[:, :V].double()).argmax(1)[:, None]
    col = torch.arange(K + 1, device=z.device)[None, :]
    padded = torch.cat([ids, ids[:, :1]], 1)
    tokens = torch.where(col < n[:, None], padded, torch.where(col == n[:, None], new, -torch.ones_like(padded)))
    return tokens.to(torch.int32), n.to(torch.int32)


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    s, lens = prepare(case, seed), _lens(case)
    if case["op"] == "packed":
        G, dh, w = case["H"] // case["Hkv"], case["dh"], case["window"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        a = 0
        for L in lens:
            for lo in range(0, L, 1024):                                # some query rows at a time
                hi = min(L, lo + 1024)
                i = torch.arange(lo, hi, device="cuda")[:, None]
                first = max(0, lo - w + 1) if w else 0
                j = torch.arange(first, hi, device="cuda")[None, :]
                hidden = (j > i) | (j <= i - w if w else j < 0)
                for h in range(case["H"]):
                    k = s["k"][a + first:a + hi, h // G].double()
                    v = s["v"][a + first:a + hi, h // G].double()
                    e = s["q"][a + lo:a + hi, h].double() @ k.T / dh ** 0.5
                    e[hidden] = -float("inf")
                    out[a + lo:a + hi, h] = torch.softmax(e, 1) @ v
            a += L
        return out
    if case["op"] == "prefix":
        B, H, T, dh = s["q"].shape
        G = H // case["Hkv"]
        out = torch.empty(B, T, H, dh, dtype=torch.float64, device="cuda")
        for g in range(case["Hkv"]):
            kp, vp = s["kp"][g].double(), s["vp"][g].double()
            for b in range(B):
                k = torch.cat([kp, s["kc"][b, g, :lens[b]].double()])
                v = torch.cat([vp, s["vc"][b, g, :lens[b]].double()])
                e = s["q"][b, g * G:(g + 1) * G].double() @ k.T / dh ** 0.5          # [G, T, keys]
                hidden = torch.arange(k.shape[0], device="cuda")[None, :] > k.shape[0] - T + torch.arange(T, device="cuda")[:, None]
                e[hidden.expand_as(e)] = -float("inf")
                out[b, :, g * G:(g + 1) * G] = (torch.softmax(e, -1) @ v).transpose(0, 1)
        return out.reshape(B, T, H * dh)
    B, K, V, temp = case["B"], case["K"], case["V"], case["temperature"]
    tokens = torch.full((B, K + 1), -1, dtype=torch.int32)
    count = torch.zeros(B, dtype=torch.int32)
    draft, u = s["draft"].tolist(), s["u"].double().tolist()
    for b in range(B):
        weights = None
        for i in range(lens[b] + 1):
            z = s["target"][b * (K + 1) + i, :V].double()
            if temp == 0:
                best = int((z == z.max()).nonzero()[0, 0])
                tokens[b, i] = best
                if i < lens[b] and draft[b][i] == best:
                    count[b] += 1
                    continue
                break
            p = torch.exp((z - z.max()) / temp)
            p = p / p.sum()
            if i == lens[b]:
                weights = p
                break
            y = s["draft_logits"][b * K + i, :V].double()
            q = torch.exp((y - y.max()) / temp)
            q = q / q.sum()
            x = draft[b][i]
            if u[b][i] * float(q[x]) < float(p[x]):
                tokens[b, i] = x
                count[b] += 1
                continue
            weights = torch.relu(p - q)
            break
        if weights is not None:
            score = weights / s["noise"][b, :V].double()
            tokens[b, int(count[b])] = int((score == score.max()).nonzero()[0, 0])
    return tokens, count
