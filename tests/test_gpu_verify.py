"""Verification of drafted tokens on the GPU (tfm_verify_draft) against its plain form in 64 bits: equal tokens
and counts; and that the answers are distributed as the target's own."""
import numpy as np
import pytest

from batch_ref import verify

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from decoder_only_transformer_gb300 import tfm  # noqa: E402

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    tfm.load()
    yield
    tfm.device_status()


def _inputs(seed, B, K, V, ld=None, std=2.0, off=0.6):
    g = torch.Generator().manual_seed(seed)
    ld = ld or (V + 3) // 4 * 4
    target = torch.randn(B * (K + 1), ld, generator=g) * std
    dl = target.view(B, K + 1, ld)[:, :K].reshape(B * K, ld) + off * torch.randn(B * K, ld, generator=g)
    noise = torch.empty(B, ld).exponential_(generator=g).clamp_(min=1e-30)
    draft = torch.zeros(B, K, dtype=torch.int32)
    if K:
        race = torch.empty(B * K, V).exponential_(generator=g)
        draft = (dl[:, :V].softmax(1) / race).argmax(1).view(B, K).int()
    u = torch.rand(B, K, generator=g)
    return [t.cuda() for t in (target, dl, draft, u, noise)]


def _call(target, dl, draft, u, noise, V, n_draft=None, temperature=1.0):
    B, K = draft.shape
    ws = torch.full((tfm.verify_draft_workspace_bytes(B, K, V),), 255, dtype=torch.uint8, device="cuda")
    tokens = torch.full((B, K + 1), -9, dtype=torch.int32, device="cuda")
    acc = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    nd = None if n_draft is None else torch.tensor(n_draft, dtype=torch.int32).cuda()
    tfm.verify_draft(target, dl, draft, nd, u, noise, V, tokens, acc, ws, temperature=temperature)
    torch.cuda.synchronize()
    return tokens.cpu().numpy(), acc.cpu().numpy()


def _same(got, want):
    assert np.array_equal(got[1], want[1]), (got[1], want[1])
    assert np.array_equal(got[0], want[0])


@pytest.mark.parametrize("V", [1, 2, 5, 23, 255, 4095, 4096, 4097, 10000, 50257])
@pytest.mark.parametrize("B,K", [(1, 4), (9, 3), (2, 0), (3, 64)])
@pytest.mark.parametrize("temperature", [0.0, 1.0, 0.7])
def test_sizes(V, B, K, temperature):
    if K == 64 and V > 5000:
        pytest.skip("covered by the smaller ones")
    a = _inputs(V + B + K, B, K, V)
    nd = [K - (b % (K + 1)) for b in range(B)]
    _same(_call(*a, V, nd, temperature), verify(a[0], a[1], a[2], nd, a[3], a[4], V, temperature))
    _same(_call(*a, V, None, temperature), verify(a[0], a[1], a[2], [K] * B, a[3], a[4], V, temperature))


def test_padding_columns_do_not_count():
    V, B, K = 4099, 4, 3
    a = _inputs(1, B, K, V, ld=4112)
    want = verify(a[0], a[1], a[2], [K] * B, a[3], a[4], V, 1.0)
    for t in (a[0], a[1]):
        t[:, V:] = 1e9
    a[4][:, V:] = 1e-30
    _same(_call(*a, V), want)
    _same(_call(*a, V, temperature=0.0), verify(a[0], None, a[2], [K] * B, None, None, V, 0))


def test_greedy_needs_the_target_alone_and_ties_go_to_the_lowest():
    V, B, K = 9000, 3, 2
    target = torch.zeros(B * (K + 1), V, device="cuda")
    target[:, 5000] = 3.0
    target[:, 4500] = 3.0
    draft = torch.tensor([[4500, 4500], [4500, 5000], [5000, 4500]], dtype=torch.int32, device="cuda")
    tokens, n = _call(target, None, draft, None, None, V, temperature=0.0)
    assert n.tolist() == [2, 1, 0]
    assert tokens.tolist() == [[4500, 4500, 4500], [4500, 4500, -1], [4500, -1, -1]]


def test_race_ties_go_to_the_lowest():
    V = 9000
    target = torch.zeros(1, V, device="cuda")
    noise = torch.ones(1, V, device="cuda")
    noise[0, [8000, 300, 5000]] = 0.5
    tokens, n = _call(target, torch.empty(0, V, device="cuda"), torch.empty(1, 0, dtype=torch.int32, device="cuda"),
                      torch.empty(1, 0, device="cuda"), noise, V)
    assert tokens.tolist() == [[300]] and n.tolist() == [0]


def test_close_races_are_decided_in_64_bits():
    """Weights apart by a few 2^-24: fp32 cannot order them, the answer is still the definition's."""
    V, B = 8200, 64
    g = torch.Generator().manual_seed(5)
    target = torch.randn(B, V, generator=g) * 0.01
    noise = torch.full((B, V), 1.0)
    top = torch.randint(0, V, (B, 6), generator=g)
    for j in range(6):                                  # six tokens of nearly equal weight / noise
        z = 3.0 + 0.25 * j
        target[torch.arange(B), top[:, j]] = z
        exact = np.exp(z - 3.0)
        off = torch.randint(-3, 4, (B,), generator=g).double() * 2.0 ** -24
        noise[torch.arange(B), top[:, j]] = (0.125 * exact * (1 + off)).float()
    K0 = torch.empty(B, 0, dtype=torch.int32, device="cuda")
    a = target.cuda(), torch.empty(0, V, device="cuda"), K0, torch.empty(B, 0, device="cuda"), noise.cuda()
    _same(_call(*a, V), verify(a[0], a[1], a[2], [0] * B, a[3], a[4], V, 1.0))


def test_masked_and_infinite_logits():
    V, B, K = 5000, 7, 2
    target, dl, draft, u, noise = _inputs(8, B, K, V)
    t3, d3 = target.view(B, K + 1, -1), dl.view(B, K, -1)
    t3[0, 0] = -INF                                      # no token has any weight: refused, no new token
    t3[1, 0, 4000] = INF                                 # all weight on one token
    d3[1, 0, 4000] = -INF
    t3[2, 0, ::2] = NAN                                  # NaN counts as no weight
    t3[3] = -INF
    t3[3, :, 17] = -1e30                                 # a single token left, the type's low end beside it
    t3[3, :, 18] = torch.finfo(torch.float32).min
    d3[4, 0, int(draft[4, 0])] = -INF                    # the drafter gave it no weight: accepted if the target does
    t3[5, 0, int(draft[5, 0])] = -INF                    # the target gives it none: refused
    d3[6] = -INF                                         # a drafter's row without any weight
    for temp in (1.0, 0.5):
        want = verify(target, dl, draft, [K] * B, u, noise, V, temp)
        got = _call(target, dl, draft, u, noise, V, temperature=temp)
        _same(got, want)
        assert got[0][0].tolist() == [-1, -1, -1] and got[0][1][0] == 4000 and got[1][5] == 0
    _same(_call(target, dl, draft, u, noise, V, temperature=0.0), verify(target, None, draft, [K] * B, None, None, V, 0))


def test_equal_models_accept_everything_and_a_refusal_without_a_rest_draws_from_p():
    V, B, K = 3001, 5, 4
    target, dl, draft, u, noise = _inputs(9, B, K, V, off=0.0)
    tokens, n = _call(target, dl, draft, u, noise, V)
    assert n.tolist() == [K] * B and np.array_equal(tokens[:, :K], draft.cpu().numpy())
    u[:] = 2.0                                           # out of [0, 1): refused although p = q
    _same(_call(target, dl, draft, u, noise, V), verify(target, dl, draft, [K] * B, u, noise, V, 1.0))


def test_ids_and_counts_out_of_range():
    V, B, K = 500, 3, 2
    a = _inputs(10, B, K, V)
    a[2][1, 0] = V
    a[2][2, 0] = -1
    for temp in (1.0, 0.0):
        _same(_call(*a, V, temperature=temp), verify(a[0], a[1], a[2], [K] * B, a[3], a[4], V, temp))
        with pytest.raises(tfm.TfmError) as e:
            tfm.device_status()
        assert e.value.status == tfm.TFM_EBADTOKEN
    a = _inputs(10, B, K, V)
    _same(_call(*a, V, [3, -1, 1]), verify(*a[:3], [2, 0, 1], *a[3:], V, 1.0))
    with pytest.raises(tfm.TfmError) as e:
        tfm.device_status()
    assert e.value.status == tfm.TFM_EINVAL


def test_answers_are_distributed_as_the_targets():
    """First token of many runs with the same two models against the target's probabilities: each count is binomial,
    6 standard deviations of its own (and 6 for rare ones) bound it."""
    V, B = 12, 20000
    g = torch.Generator().manual_seed(3)
    z, y = torch.randn(V, generator=g) * 1.5, torch.randn(V, generator=g) * 1.5
    p, q = z.double().softmax(0), y.double().softmax(0)
    target = z.repeat(B * 2, 1).cuda()
    dl = y.repeat(B, 1).cuda()
    draft = torch.multinomial(q, B, replacement=True, generator=g).int().view(B, 1).cuda()
    u = torch.rand(B, 1, generator=g).cuda()
    noise = torch.empty(B, V).exponential_(generator=g).clamp_(min=1e-30).cuda()
    tokens, n = _call(target, dl, draft, u, noise, V)
    count = np.bincount(tokens[:, 0], minlength=V)
    sd = np.sqrt(B * p.numpy() * (1 - p.numpy()))
    assert (np.abs(count - B * p.numpy()) <= 6 * sd + 6).all()
    rate = float(torch.minimum(p, q).sum())
    assert abs(n.mean() - rate) <= 6 * np.sqrt(rate * (1 - rate) / B)


def test_graph_replay_and_repeats_agree():
    V, B, K = 20000, 6, 3
    target, dl, draft, u, noise = _inputs(12, B, K, V)
    ws = torch.empty(tfm.verify_draft_workspace_bytes(B, K, V), dtype=torch.uint8, device="cuda")
    tokens = torch.empty(B, K + 1, dtype=torch.int32, device="cuda")
    acc = torch.empty(B, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        tfm.verify_draft(target, dl, draft, None, u, noise, V, tokens, acc, ws)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            tfm.verify_draft(target, dl, draft, None, u, noise, V, tokens, acc, ws)
    for seed in (12, 13, 14):
        new = _inputs(seed, B, K, V)
        for old, t in zip((target, dl, draft, u, noise), new):
            old.copy_(t)
        for _ in range(3):
            tokens.fill_(-9)
            g.replay()
            torch.cuda.synchronize()
            _same((tokens.cpu().numpy(), acc.cpu().numpy()), verify(*new[:3], [K] * B, *new[3:], V, 1.0))


@pytest.mark.parametrize("B", [4, 100])                 # the race's CTAs decide, or a launch before it
@pytest.mark.parametrize("V", [600, 9001])
def test_acceptance_on_the_verge(B, V):
    """u q(x) within 2e-5 of p(x): closer than fp32 can tell, further than the fp32 sums are off (5e-6)."""
    K = 3
    target, dl, draft, u, noise = _inputs(B + V, B, K, V, off=0.2)
    p = (target[:, :V].double().softmax(1)).view(B, K + 1, V)[:, :K].gather(2, draft[..., None].long())[..., 0]
    q = (dl[:, :V].double().softmax(1)).view(B, K, V).gather(2, draft[..., None].long())[..., 0]
    g = torch.Generator().manual_seed(V)
    side = (torch.randint(0, 2, (B, K), generator=g) * 2 - 1).cuda().double()
    u = (p / q * (1 + 2e-5 * side)).float()
    u = torch.where(u < 1, u, torch.full_like(u, 0.25))
    want = verify(target, dl, draft, [K] * B, u, noise, V, 1.0)
    _same(_call(target, dl, draft, u, noise, V), want)
    assert 0 < want[1].sum() < B * K


@pytest.mark.parametrize("B", [4, 90])
@pytest.mark.parametrize("refused", [False, True])
def test_close_races_of_few_and_many(B, refused):
    """Six tokens 3e-5 apart, with and without a refused row: closer than fp32 can tell (its bound is 2.5e-5 of
    p + q on each side), further than the fp32 sums of both rows, 1.4e-6 each, move p - q against one another
    (p / (p - q) stays below 4 among the largest weights: 1.1e-5)."""
    V, K = 8300, 1 if refused else 0
    g = torch.Generator().manual_seed(B)
    target = (torch.randn(B * (K + 1), V, generator=g) * 0.1).cuda()
    dl = (torch.randn(B * K, V, generator=g) * 0.1 - 1).cuda()
    draft = torch.zeros(B, K, dtype=torch.int32, device="cuda")
    u = torch.ones(B, K, device="cuda")
    if refused:                                         # p(0) = 0: always refused
        target[0::2, 0] = -INF
    noise = torch.full((B, V), 30.0, device="cuda")
    rows = target.view(B, K + 1, V)[:, 0, :].double()
    w = rows.softmax(1)
    if refused:
        w = (w - dl[:, :V].double().softmax(1)).clamp(min=0)
    for b in range(B):
        top = torch.argsort(w[b], descending=True)[torch.randperm(200, generator=g)[:6]]
        noise[b, top] = (w[b, top] * 4000 * (1 + 3e-5 * torch.randperm(6, generator=g).cuda().double())).float()
    want = verify(target, dl if K else None, draft, [K] * B, u if K else None, noise, V, 1.0)
    got = _call(target, dl if K else torch.empty(0, V, device="cuda"), draft, u, noise, V)
    _same(got, want)
