"""The batched-serving operators as a serving program uses them, together: a batch of prompts prefilled at once,
then steps that score drafted tokens over the shared prefix and the own caches and keep what the verification
accepts.  And the calls around that: other streams, two at once, graphs that share a workspace, the smallest and
the largest sizes."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest

from batch_ref import bound, f64, packed, prefix, verify

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from decoder_only_transformer_gb300 import tfm  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tfm.load()
    yield
    tfm.device_status()


def _bytes(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def _norm(t):
    return float(np.sqrt((f64(t) ** 2).sum(-1).max(initial=0.0)))


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
@pytest.mark.parametrize("temperature", [0.0, 0.8])
@pytest.mark.parametrize("H,Hkv,dh", [(8, 2, 64), (4, 4, 32), (4, 1, 128)])
def test_serving_run(H, Hkv, dh, temperature, graph):
    B, P, K, V, room, steps = 4, 150, 3, 1003, 130, 4
    T, ld = K + 1, 1004
    g = torch.Generator(device="cuda").manual_seed(H * dh)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
    table, places = rand(V, H + 2 * Hkv, dh), rand(P + room, H + 2 * Hkv, dh)
    w_out, big = rand(H * dh, ld) * (H * dh) ** -0.5, 3 * rand(V, ld)

    def qkv(tokens, first=0):
        """The fused projection's rows of tokens that stand at first, first + 1, ..."""
        return (table[tokens] + places[first:first + len(tokens)]).to(torch.bfloat16)

    def logits(o, tokens):
        return o.float() @ w_out + big[tokens]

    # Prompts that begin alike; one is the shared part alone.
    shared = torch.randint(0, V, (P,), device="cuda", generator=g)
    texts = [torch.cat([shared, torch.randint(0, V, (n,), device="cuda", generator=g)]) for n in (5, 0, 70, 64)]

    def prefill():
        x = torch.cat([qkv(t) for t in texts])
        lens = [len(t) for t in texts]
        q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
        o = torch.empty(len(x), H, dh, dtype=torch.bfloat16, device="cuda")
        tfm.packed_attention(q, k, v, o, _ints(np.cumsum([0] + lens)),
                             _bytes(tfm.packed_attention_workspace_bytes(len(x), B)))
        ref = packed(q, k, v, lens)
        tol = bound(f64(v), dh, max(lens), _norm(q) * _norm(k) * dh ** -0.5, torch.bfloat16)
        assert np.abs(f64(o) - ref).max() <= tol
        return q, k, v, o, lens, ref, tol

    _, k, v, o, lens, _, _ = prefill()
    kp, vp = (t[:P].transpose(0, 1).contiguous() for t in (k, v))
    kc, vc = (torch.full((B, Hkv, room, dh), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for b in range(B):
        a = sum(lens[:b])
        for cache, rows in ((kc, k), (vc, v)):
            cache[b, :, :lens[b] - P] = rows[a + P:a + lens[b]].transpose(0, 1)
    last = np.cumsum(lens) - 1
    new = [int(i) for i in logits(o[last].reshape(B, -1), torch.stack([t[-1] for t in texts]))[:, :V].argmax(1)]

    # What a step works on stays where it is, so that one recorded graph serves all steps.
    q = torch.empty(B, H, T, dh, dtype=torch.bfloat16, device="cuda")
    o = torch.empty(B, T, H * dh, dtype=torch.bfloat16, device="cuda")
    own, ids = _ints([0] * B), torch.zeros(B, T, dtype=torch.int64, device="cuda")
    draft, u = torch.zeros(B, K, dtype=torch.int32, device="cuda"), torch.zeros(B, K, device="cuda")
    noise, dlogits = torch.ones(B, ld, device="cuda"), torch.zeros(B * K, ld, device="cuda")
    target = torch.zeros(B * T, ld, device="cuda")
    tokens, accepted = torch.zeros(B, T, dtype=torch.int32, device="cuda"), _ints([0] * B)
    ws = _bytes(max(tfm.prefix_attention_workspace_bytes(B, H, Hkv, T, dh), tfm.verify_draft_workspace_bytes(B, K, V)))

    def step():
        tfm.prefix_attention(q, kp, vp, kc, vc, o, own, ws)
        target.copy_(logits(o.view(B * T, -1), ids.view(-1)))
        tfm.verify_draft(target, dlogits, draft, None, u, noise, V, tokens, accepted, ws, temperature=temperature)

    if graph:
        kc.zero_(), vc.zero_(), q.zero_()                # nothing to see in the warm-up
        kc_, vc_ = kc.clone(), vc.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        recorded = torch.cuda.CUDAGraph()
        with torch.cuda.graph(recorded):
            step()
        assert torch.equal(kc, kc_) and torch.equal(vc, vc_)
        for b in range(B):
            a = sum(lens[:b])
            for cache, rows in ((kc, k), (vc, v)):
                cache[b, :, :lens[b] - P] = rows[a + P:a + lens[b]].transpose(0, 1)
        step = recorded.replay

    outs, kept = [[] for _ in range(B)], 0
    n_own = [len(t) - P for t in texts]
    for _ in range(steps):
        u.uniform_(generator=g)
        noise.exponential_(generator=g).clamp_(min=1e-30)
        for b in range(B):
            ids[b, 0] = new[b]
            for i in range(K):                           # the drafter: what follows a token, without the text
                z = big[ids[b, i], :V]
                ids[b, i + 1] = ((z / (temperature or 0.1)).softmax(0) /
                                 torch.empty(V, device="cuda").exponential_(generator=g)).argmax()
            x = qkv(ids[b], P + n_own[b])
            q[b] = x[:, :H].transpose(0, 1)
            kc[b, :, n_own[b]:n_own[b] + T] = x[:, H:H + Hkv].transpose(0, 1)
            vc[b, :, n_own[b]:n_own[b] + T] = x[:, H + Hkv:].transpose(0, 1)
        draft.copy_(ids[:, 1:])
        dlogits.copy_(big[ids[:, :K]].view(B * K, ld))
        own.copy_(_ints([n + T for n in n_own]))
        step()
        torch.cuda.synchronize()
        want = verify(target, dlogits, draft, [K] * B, u, noise, V, temperature)
        assert np.array_equal(accepted.cpu().numpy(), want[1])
        assert np.array_equal(tokens.cpu().numpy(), want[0])
        for b, n in enumerate(want[1]):
            texts[b] = torch.cat([texts[b], ids[b, :n + 1]])
            outs[b].append(o[b, :n + 1].clone())
            n_own[b] += int(n) + 1
            new[b] = int(want[0][b, n])
            kept += int(n)
    assert 0 < kept < B * K * steps                      # some were accepted, some refused

    # The texts that came out, prefilled at once, agree with what the steps saw.
    _, _, _, _, lens, ref, tol = prefill()
    for b in range(B):
        rows = torch.cat(outs[b])
        a = sum(lens[:b + 1]) - len(rows)
        assert np.abs(f64(rows) - ref[a:a + len(rows)].reshape(len(rows), -1)).max() <= tol


def _packed_inputs(seed, T, H, Hkv, dh):
    g = torch.Generator().manual_seed(seed)
    r = lambda h: torch.randn(T, h, dh, generator=g).to(torch.bfloat16).cuda()
    return r(H), r(Hkv), r(Hkv)


def _prefix_inputs(seed, B, H, Hkv, T, P, room, dh):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
    return r(B, H, T, dh), r(Hkv, P, dh), r(Hkv, P, dh), r(B, Hkv, room, dh), r(B, Hkv, room, dh)


def _verify_inputs(seed, B, K, V, ld):
    g = torch.Generator().manual_seed(seed)
    target = torch.randn(B * (K + 1), ld, generator=g) * 2
    dl = target.view(B, K + 1, ld)[:, :K].reshape(B * K, ld) + 0.5 * torch.randn(B * K, ld, generator=g)
    draft = torch.randint(0, V, (B, K), generator=g).int()
    if K:
        draft[:, 0] = dl.view(B, K, ld)[:, 0, :V].argmax(1).int()
    return [t.cuda() for t in (target, dl, draft, torch.rand(B, K, generator=g),
                               torch.empty(B, ld).exponential_(generator=g).clamp_(min=1e-30))]


def _calls(seed):
    """A call of each operator, with buffers and a workspace of its own: (run(stream), its outputs)."""
    q, k, v = _packed_inputs(seed, 700, 4, 2, 64)
    cu, o1 = _ints([0, 300, 300, 640]), torch.empty_like(q)
    w1 = _bytes(tfm.packed_attention_workspace_bytes(700, 3))
    a = _prefix_inputs(seed + 1, 5, 8, 2, 3, 500, 90, 128)
    lens, o2 = _ints([90, 3, 64, 17, 0]), torch.empty(5, 3, 1024, dtype=torch.bfloat16, device="cuda")
    w2 = _bytes(tfm.prefix_attention_workspace_bytes(5, 8, 2, 3, 128))
    t = _verify_inputs(seed + 2, 6, 4, 20000, 20000)
    tokens, n = _ints([[0] * 5] * 6), _ints([0] * 6)
    w3 = _bytes(tfm.verify_draft_workspace_bytes(6, 4, 20000))
    runs = (lambda s=None, w=w1: tfm.packed_attention(q, k, v, o1, cu, w, stream=s),
            lambda s=None, w=w2: tfm.prefix_attention(*a, o2, lens, w, stream=s),
            lambda s=None, w=w3: tfm.verify_draft(t[0], t[1], t[2], None, t[3], t[4], 20000, tokens, n, w, stream=s))
    o1.zero_()
    return runs, (o1, o2, tokens, n), (w1, w2, w3)


def _outputs(outs):
    torch.cuda.synchronize()
    return [o.clone() for o in outs]


def _clear(outs):
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()


def test_given_stream_and_two_calls_at_once():
    """The calls of two sets on two streams, in turn and many at once, leave what each left alone."""
    sets, want = [_calls(1), _calls(50)], []
    for runs, outs, _ in sets:
        for run in runs:
            run()
        want.append(_outputs(outs))
        _clear(outs)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for (runs, _, _), s in zip(sets, streams):
            for run in runs:
                run(s)
    for (_, outs, _), w in zip(sets, want):
        for got, ref in zip(_outputs(outs), w):
            assert torch.equal(got, ref)


def test_graphs_that_share_a_workspace():
    """Graphs of different calls with one workspace, replayed one behind the other on a stream in any order."""
    sets = [_calls(3), _calls(60)]
    ws = _bytes(max(w.numel() for _, _, all_ws in sets for w in all_ws))
    want, graphs = [], []
    for runs, outs, _ in sets:
        for run in runs:
            run()
        want.append(_outputs(outs))
        for run in runs:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                run(None, ws)
            graphs.append(graph)
        _clear(outs)
    for i in [0, 1, 2, 3, 4, 5, 5, 2, 4, 1, 3, 0, 0, 5, 1, 4]:
        graphs[i].replay()
    for (_, outs, _), w in zip(sets, want):
        for got, ref in zip(_outputs(outs), w):
            assert torch.equal(got, ref)


def test_nothing_to_do():
    """Sizes of zero: no row, no sequence, no batch, nothing drafted, no prefix memory."""
    for dtype in (torch.bfloat16, torch.float32):
        z = torch.empty(0, 4, 64, dtype=dtype, device="cuda")
        tfm.packed_attention(z, z, z, z, _ints([0, 0, 0]), _bytes(tfm.packed_attention_workspace_bytes(0, 2)))
        x = torch.randn(5, 4, 64, device="cuda").to(dtype)
        o = torch.full_like(x, 7.0)
        tfm.packed_attention(x, x, x, o, _ints([0]), _bytes(tfm.packed_attention_workspace_bytes(5, 0)))
        tfm.packed_attention(x, x, x, o, _ints([3, 3, 3]), _bytes(tfm.packed_attention_workspace_bytes(5, 2)))
        torch.cuda.synchronize()
        assert (o == 7.0).all()
    e = torch.empty(0, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    a = _prefix_inputs(5, 2, 4, 2, 1, 1, 6, 64)
    tfm.prefix_attention(e, a[1], a[2], a[3], a[4], e.view(0, 1, 256), _ints([]),
                         _bytes(tfm.prefix_attention_workspace_bytes(0, 4, 2, 1, 64)))
    none = torch.empty(2, 0, 64, dtype=torch.bfloat16, device="cuda")
    o = torch.full((2, 1, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    tfm.prefix_attention(a[0], none, none, a[3], a[4], o, _ints([6, 0]),
                         _bytes(tfm.prefix_attention_workspace_bytes(2, 4, 2, 1, 64)))
    ref = prefix(a[0], a[1], a[2], a[3], a[4], [6, 0], 0)
    tol = bound(f64(a[4]), 64, 6, _norm(a[0]) * _norm(a[3]) / 8, torch.bfloat16)
    assert np.abs(f64(o) - ref).max() <= tol and (o[1] == 0).all()
    t = torch.randn(0, 8, device="cuda")
    tfm.verify_draft(t, t, _ints([]).view(0, 3), None, t.view(0, 8)[:, :3], t, 8, _ints([]), _ints([]),
                     _bytes(tfm.verify_draft_workspace_bytes(0, 3, 8)))
    tfm.device_status()


def test_equal_tensors_and_offsets_in_a_larger_array():
    """q, k and v one tensor; offsets that begin in the middle of an array of them."""
    x = torch.randn(300, 4, 64, device="cuda").to(torch.bfloat16)
    o = torch.full_like(x, 7.0)
    offsets = _ints([1, 2, 0, 10, 10, 200])
    tfm.packed_attention(x, x, x, o, offsets[3:], _bytes(tfm.packed_attention_workspace_bytes(300, 2)))
    y = x[10:200]
    assert np.abs(f64(o[10:200]) - packed(y, y, y, [0, 190])).max() <= \
        bound(f64(y), 64, 190, _norm(y) ** 2 / 8, torch.bfloat16)
    assert (o[:10] == 7.0).all() and (o[200:] == 7.0).all()


def test_many_sequences_and_heads():
    """More sequences than rows of a plan, most of them empty; an odd number of many heads."""
    rng = np.random.default_rng(3)
    lens = np.zeros(70000, np.int64)
    lens[rng.choice(70000, 400, replace=False)] = rng.integers(1, 6, 400)
    T = int(lens.sum())
    for dtype in (torch.bfloat16, torch.float32):
        q, k, v = (t.to(dtype) for t in _packed_inputs(8, T, 4, 2, 32))
        o = torch.zeros_like(q)
        tfm.packed_attention(q, k, v, o, _ints(np.cumsum([0] + list(lens))),
                             _bytes(tfm.packed_attention_workspace_bytes(T, len(lens))))
        ref = packed(q, k, v, [int(n) for n in lens if n])
        assert np.abs(f64(o) - ref).max() <= bound(f64(v), 32, 5, _norm(q) * _norm(k) * 32 ** -0.5, dtype)
    q, k, v = _packed_inputs(9, 140, 259, 37, 32)
    o = torch.zeros_like(q)
    tfm.packed_attention(q, k, v, o, _ints([0, 1, 140]), _bytes(tfm.packed_attention_workspace_bytes(140, 2)))
    assert np.abs(f64(o) - packed(q, k, v, [1, 139])).max() <= \
        bound(f64(v), 32, 139, _norm(q) * _norm(k) * 32 ** -0.5, torch.bfloat16)


@pytest.mark.parametrize("B,H,Hkv,T", [(4096, 2, 1, 1), (300, 16, 1, 8), (2, 128, 1, 1), (1, 1, 1, 128)])
def test_largest_batches_of_a_step(B, H, Hkv, T):
    """B at its limit with caches of a few tokens; (H / Hkv) T at its limit."""
    rng = np.random.default_rng(B)
    lens = [int(n) for n in rng.integers(0, 9, B)]
    a = _prefix_inputs(B + H, B, H, Hkv, T, 70, 140, 32)
    if T == 128:
        lens = [130]
    o = torch.empty(B, T, H * 32, dtype=torch.bfloat16, device="cuda")
    tfm.prefix_attention(*a, o, _ints(lens), _bytes(tfm.prefix_attention_workspace_bytes(B, H, Hkv, T, 32)))
    tol = bound(np.concatenate([f64(a[2]).ravel(), f64(a[4]).ravel()]), 32, 70 + max(lens),
                _norm(a[0]) * max(_norm(a[1]), _norm(a[3])) * 32 ** -0.5, torch.bfloat16)
    some = sorted({0, B // 2, B - 1})
    ref = prefix(a[0][some], a[1], a[2], a[3][some], a[4][some], [lens[b] for b in some], 70)
    assert torch.isfinite(o).all()
    assert np.abs(f64(o[some]) - ref).max() <= tol
    # a sequence's answer does not depend on the batch it is in, up to both sides' roundings
    for b in some:
        one = torch.empty(1, T, H * 32, dtype=torch.bfloat16, device="cuda")
        tfm.prefix_attention(a[0][b:b + 1], a[1], a[2], a[3][b:b + 1], a[4][b:b + 1], one, _ints([lens[b]]),
                             _bytes(tfm.prefix_attention_workspace_bytes(1, H, Hkv, T, 32)))
        assert np.abs(f64(one[0]) - f64(o[b])).max() <= 2 * tol


def test_caches_of_a_larger_pool():
    """More sequences in the caches than in the call: the first B are meant."""
    a = _prefix_inputs(21, 6, 4, 2, 2, 33, 20, 64)
    lens = [20, 2, 7]
    o = torch.full((3, 2, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    tfm.prefix_attention(a[0][:3], *a[1:], o, _ints(lens), _bytes(tfm.prefix_attention_workspace_bytes(3, 4, 2, 2, 64)),
                         prefix_len=30)
    ref = prefix(a[0][:3], a[1], a[2], a[3][:3], a[4][:3], lens, 30)
    v = np.concatenate([f64(a[2]).ravel(), f64(a[4]).ravel()])
    assert np.abs(f64(o) - ref).max() <= bound(v, 64, 50, _norm(a[0]) * max(_norm(a[1]), _norm(a[3])) / 8, torch.bfloat16)


@pytest.mark.parametrize("B,K,V,temperature", [(2, 64, 10000, 1.0), (1, 64, 50257, 0.7), (1, 64, 50257, 0.0),
                                               (700, 1, 40, 1.0), (3000, 0, 9, 0.9), (1, 1, 1 << 20, 1.0),
                                               (3, 2, 300, 1e-30), (3, 2, 300, 1e30), (3, 2, 300, 1e-4)])
def test_largest_verifications(B, K, V, temperature):
    ld = (V + 3) // 4 * 4
    a = _verify_inputs(V + K, B, K, V, ld)
    tokens, n = _ints([[-9] * (K + 1)] * B), _ints([-9] * B)
    ws = torch.full((tfm.verify_draft_workspace_bytes(B, K, V),), 255, dtype=torch.uint8, device="cuda")
    tfm.verify_draft(a[0], a[1], a[2], None, a[3], a[4], V, tokens, n, ws, temperature=temperature)
    t = float(np.float32(temperature))
    want = verify(a[0], a[1], a[2], [K] * B, a[3], a[4], V, t)
    assert np.array_equal(n.cpu().numpy(), want[1]) and np.array_equal(tokens.cpu().numpy(), want[0])


@pytest.mark.parametrize("kwargs", [dict(temperature=1e-31), dict(temperature=1e31), dict(vocab=(1 << 24) + 1)])
def test_refused_verifications(kwargs):
    a = _verify_inputs(1, 2, 2, 64, 64)
    call = dict(vocab=64, temperature=1.0)
    call.update(kwargs)
    with pytest.raises((ValueError, tfm.TfmError)):
        tfm.verify_draft(a[0], a[1], a[2], None, a[3], a[4], call["vocab"], _ints([[0] * 3] * 2), _ints([0, 0]),
                         _bytes(1 << 16), temperature=call["temperature"])


def test_offsets_beyond_32_bits():
    """Rows more than 2^32 elements into their arrays, values that are not finite among them."""
    far = (1 << 32) + 4096
    buf = torch.empty(far + (1 << 16), dtype=torch.bfloat16, device="cuda")
    T, dh = 140, 64
    view = lambda at: buf[at:].as_strided((T, 2, dh), (dh, far, 1))
    q, k, v, o = (view(i * T * dh) for i in range(4))
    for t, x in zip((q, k, v), _packed_inputs(31, T, 2, 2, dh)):
        t.copy_(x)
    o.fill_(7.0)
    clean, tol = packed(q, k, v, [5, 130]), bound(f64(v), dh, 130, _norm(q.contiguous()) * _norm(k.contiguous()) / 8, torch.bfloat16)
    v[100, 1, 3] = float("inf")
    tfm.packed_attention(q, k, v, o, _ints([0, 5, 135]), _bytes(tfm.packed_attention_workspace_bytes(T, 2)))
    got = f64(o)
    seen = np.zeros_like(clean, bool)
    seen[100:, 1, 3] = True
    assert np.abs(got[:135] - clean)[~seen].max() <= tol
    assert np.isposinf(got[:135][seen]).all() and (got[135:] == 7.0).all()
    del buf, q, k, v, o, view

    # One long cache: the key at j outweighs all others by e^100.
    n, j = (1 << 25) + 150, (1 << 25) + 101
    kc = torch.zeros(1, 1, n, 128, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty(1, 1, n, 128, dtype=torch.bfloat16, device="cuda").normal_()
    q = torch.full((1, 1, 1, 128), 1.0, dtype=torch.bfloat16, device="cuda")
    kc[0, 0, j] = 1.0
    o = torch.empty(1, 1, 128, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(1, 0, 128, dtype=torch.bfloat16, device="cuda")
    tfm.prefix_attention(q, none, none, kc, vc, o, _ints([n - 7]),
                         _bytes(tfm.prefix_attention_workspace_bytes(1, 1, 1, 1, 128)), scale=100 / 128)
    assert torch.equal(o[0, 0], vc[0, 0, j])
    del kc, vc

    # Logits whose rows lie 2^29 elements apart.
    K, V, ld = 8, 500, 1 << 29
    rows = torch.empty((K + 1) * ld, device="cuda").as_strided((K + 1, V), (ld, 1))
    a = _verify_inputs(33, 1, K, V, V)
    a[2][:] = a[1][:, :V].argmax(1).int()
    rows.copy_(a[0])
    tokens, m = _ints([[0] * (K + 1)]), _ints([0])
    tfm.verify_draft(rows, a[1], a[2], None, a[3] * 0.01, a[4], V, tokens, m,
                     _bytes(tfm.verify_draft_workspace_bytes(1, K, V)))
    want = verify(a[0], a[1], a[2], [K], a[3] * 0.01, a[4], V, 1.0)
    assert want[1][0] == K and np.array_equal(tokens.cpu().numpy(), want[0])


FIRST = """
import torch
from decoder_only_transformer_gb300 import tfm
r = lambda *s: torch.randn(*s, device="cuda")
ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
b = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")
q, cu = r(300, {H}, 64).to(torch.{dtype}), ints([0, 120, 300])
o1, w1 = torch.zeros_like(q), b(tfm.packed_attention_workspace_bytes(300, 2))
x, kp, kc = (r(*s).bfloat16() for s in ((3, 8, 2, 64), (2, 100, 64), (3, 2, 50, 64)))
o2, lens, w2 = torch.zeros(3, 2, 512, dtype=torch.bfloat16, device="cuda"), ints([50, 2, 9]), b(tfm.prefix_attention_workspace_bytes(3, 8, 2, 2, 64))
t, d, draft, u, e = r({B} * 3, 5000), r({B} * 2, 5000), ints([[1, 2]] * {B}), torch.rand({B}, 2, device="cuda"), r({B}, 5000).abs() + 0.01
tok, n, w3 = ints([[0] * 3] * {B}), ints([0] * {B}), b(tfm.verify_draft_workspace_bytes({B}, 2, 5000))
def run():
    tfm.packed_attention(q, q, q, o1, cu, w1)
    tfm.prefix_attention(x, kp, kp, kc, kc, o2, lens, w2)
    tfm.verify_draft(t, d, draft, None, u, e, 5000, tok, n, w3, temperature={temperature})
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    run()
g.replay()
torch.cuda.synchronize()
first = [z.clone() for z in (o1, o2, tok, n)]
run()
torch.cuda.synchronize()
assert all(torch.equal(a, c) for a, c in zip(first, (o1, o2, tok, n))) and o1.abs().sum() > 0 and o2.abs().sum() > 0
tfm.device_status()
print("same")
"""


@pytest.mark.parametrize("H,dtype,B,temperature", [(4, "bfloat16", 3, 1.0), (64, "bfloat16", 100, 1.0), (4, "float32", 3, 0.0)])
def test_first_calls_of_a_process_are_captured(H, dtype, B, temperature):
    """Nothing has to run before a capture: a fresh process records its first call of each operator."""
    code = FIRST.format(H=H, dtype=dtype, B=B, temperature=temperature)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]


def test_threads_on_streams_of_their_own():
    """Calls from two host threads at once, each with its stream and workspaces."""
    sets = [_calls(5), _calls(70)]
    want = []
    for runs, outs, _ in sets:
        for run in runs:
            run()
        want.append(_outputs(outs))
        _clear(outs)
    errors = []

    def work(runs):
        try:
            stream = torch.cuda.Stream()
            for _ in range(30):
                for run in runs:
                    run(stream)
        except Exception as e:                          # shown by the assertion below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(runs,)) for runs, _, _ in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for (_, outs, _), w in zip(sets, want):
        for got, ref in zip(_outputs(outs), w):
            assert torch.equal(got, ref)
