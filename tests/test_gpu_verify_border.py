"""Verification of drafted tokens where decisions stand on the border: sides that differ by a rounding of an input and no
more.  Sums in fp32 get part of them wrong, which every test shows for its own inputs; the kernel's answers have to be
those of 64 bits, whose own error (1e-15) is far below the smallest distance there is here."""
import numpy as np
import pytest

from batch_ref import verify

torch = pytest.importorskip("torch")

from decoder_only_transformer_gb300 import tfm  # noqa: E402

INF = float("inf")


def _call(target, dl, draft, u, noise, V, temperature):
    B, K = draft.shape
    ws = torch.full((tfm.verify_draft_workspace_bytes(B, K, V),), 255, dtype=torch.uint8, device="cuda")
    tokens = torch.full((B, K + 1), -9, dtype=torch.int32, device="cuda")
    acc = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    a = [t.cuda() for t in (target, dl, draft)], [t.cuda() for t in (u, noise)]
    tfm.verify_draft(*a[0], None, *a[1], V, tokens, acc, ws, temperature=temperature)
    tfm.device_status()
    return tokens.cpu().numpy(), acc.cpu().numpy()


def _same(target, dl, draft, u, noise, V, temperature):
    B, K = draft.shape
    want = verify(target, dl if K else None, draft, [K] * B, u, noise, V, float(np.float32(temperature)))
    got = _call(target, dl, draft, u, noise, V, temperature)
    assert np.array_equal(got[1], want[1]), np.flatnonzero(got[1] != want[1])
    assert np.array_equal(got[0], want[0]), np.flatnonzero((got[0] != want[0]).any(1))


def _logits(seed, B, K, V, off):
    g = torch.Generator().manual_seed(seed)
    ld = (V + 3) // 4 * 4
    target = torch.randn(B * (K + 1), ld, generator=g) * 2
    dl = target.view(B, K + 1, ld)[:, :K].reshape(B * K, ld) + off * torch.randn(B * K, ld, generator=g)
    return g, target, dl


@pytest.mark.gpu
@pytest.mark.parametrize("temperature", [1.0, 0.7, 1.3])
def test_races_of_weights_far_below_the_largest(temperature):
    """The largest weight against one e^-83 of it with as much less noise, 1e-6 apart."""
    B, V = 64, 5000
    g = torch.Generator().manual_seed(1)
    t = float(np.float32(temperature))
    target = torch.full((B, V), -INF)
    noise = torch.empty(B, V).exponential_(generator=g).clamp_(min=1e-30)
    deep = torch.randint(1, V, (B,), generator=g)
    z = -(80 + 3 * torch.rand(B, generator=g)) * temperature
    rows = torch.arange(B)
    target[:, 0], noise[:, 0] = 0.0, 0.5
    target[rows, deep] = z
    side = (torch.randint(0, 2, (B,), generator=g) * 2 - 1).double()
    noise[rows, deep] = (0.5 * torch.exp(z.double() / t) * (1 + 1e-6 * side)).float()
    assert (noise[rows, deep] > 1.2e-38).all()
    K0 = torch.empty(B, 0, dtype=torch.int32)
    want = verify(target, None, K0, [0] * B, None, noise, V, t)[0][:, 0]
    assert np.array_equal(want == 0, side.numpy() > 0)
    _same(target, torch.empty(0, V), K0, torch.empty(B, 0), noise, V, temperature)


def _probs32(z, temperature):
    """Probabilities with everything in fp32, as a kernel without a second look has them."""
    c2 = torch.tensor(1.4426950408889634, dtype=torch.float32) / temperature
    w = torch.exp2((z - z.max(1, keepdim=True).values) * c2)
    return w / w.sum(1, keepdim=True)


def _probs64(z, temperature):
    z = z.double()
    w = torch.exp((z - z.max(1, keepdim=True).values) / float(np.float32(temperature)))
    return w / w.sum(1, keepdim=True)


def _border_drafts(B, K, V, temperature):
    """u is the fp32 number nearest to p(x) / q(x) (or one further), where that is below 1."""
    g, target, dl = _logits(B + V, B, K, V, 0.3)
    draft = (dl[:, :V].softmax(1) / torch.empty(B * K, V).exponential_(generator=g)).argmax(1).view(B, K).int()
    x = draft.long()[..., None]
    rows = target.view(B, K + 1, -1)[:, :K, :V].reshape(B * K, V)
    p, q = (_probs64(z, temperature).view(B, K, V).gather(2, x)[..., 0] for z in (rows, dl[:, :V]))
    p32, q32 = (_probs32(z, temperature).view(B, K, V).gather(2, x)[..., 0] for z in (rows, dl[:, :V]))
    u = (p / q).float()
    u = u + torch.randint(-1, 2, u.shape, generator=g) * u * 2.0 ** -24
    u = torch.where(p / q < 1, u, torch.full_like(u, 0.5))
    noise = torch.empty(B, target.shape[1]).exponential_(generator=g).clamp_(min=1e-30)
    return target, dl, draft, u, noise, (u.double() * q < p), (u * q32 < p32)


@pytest.mark.parametrize("temperature", [1.0, 0.8, 1.3])
@pytest.mark.parametrize("B,K,V", [(40, 1, 9001), (200, 1, 9001), (64, 5, 20000)])
def test_border_of_acceptance_is_beyond_fp32(B, K, V, temperature):
    """What the next test stands on: plain fp32 decides some of its drafts wrongly, and both answers occur."""
    *_, want, plain = _border_drafts(B, K, V, temperature)
    assert (want != plain).sum() >= 2
    assert 0 < want.sum() < want.numel()


@pytest.mark.gpu
@pytest.mark.parametrize("temperature", [1.0, 0.8, 1.3])
@pytest.mark.parametrize("B,K,V", [(40, 1, 9001), (200, 1, 9001), (64, 5, 20000)])
def test_border_of_acceptance(B, K, V, temperature):
    target, dl, draft, u, noise, _, _ = _border_drafts(B, K, V, temperature)
    _same(target, dl, draft, u, noise, V, temperature)


def _border_races(B, V, temperature, off=1.0):
    """Token 0 is drafted and refused (p(0) = 0); among the 200 largest weights p - q six have the same weight / noise,
    up to the rounding of their noise (2^-24), and all others less."""
    g, target, dl = _logits(B + 3 * V, B, 1, V, off)
    target[0::2, 0] = -INF
    draft, u = torch.zeros(B, 1, dtype=torch.int32), torch.full((B, 1), 0.5)
    noise = torch.full((B, target.shape[1]), 30.0)
    rows = target.view(B, 2, -1)[:, 0, :V]
    w = (_probs64(rows, temperature) - _probs64(dl[:, :V], temperature)).clamp(min=0)
    for b in range(B):
        top = torch.argsort(w[b], descending=True)[torch.randperm(min(200, int((w[b] > 0).sum())), generator=g)[:6]]
        noise[b, top] = (w[b, top] / w[b].max() * 20).float()
    race = torch.where(w > 0, w / noise[:, :V].double(), torch.zeros_like(w))
    w32 = (_probs32(rows, temperature) - _probs32(dl[:, :V], temperature)).clamp(min=0)
    return target, dl, draft, u, noise, race.argmax(1), (w32 / noise[:, :V]).argmax(1)


RACES = [(40, 8300, 1.0, 1.0), (90, 8300, 1.0, 1.0), (64, 8300, 0.7, 0.3), (40, 20000, 1.3, 0.1), (6, 20000, 1.0, 1e-3)]


@pytest.mark.parametrize("B,V,temperature,off", RACES)
def test_border_of_a_race_is_beyond_fp32(B, V, temperature, off):
    *_, want, plain = _border_races(B, V, temperature, off)
    assert (want != plain).sum() >= 2


@pytest.mark.gpu
@pytest.mark.parametrize("B,V,temperature,off", RACES)
def test_border_of_a_race(B, V, temperature, off):
    target, dl, draft, u, noise, _, _ = _border_races(B, V, temperature, off)
    _same(target, dl, draft, u, noise, V, temperature)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [5, 60])
def test_refused_drafts_of_nearly_equal_models(B):
    """Rows that differ by a last bit here and there: the residual is a few 1e-7 of p in those places, nothing elsewhere, and
    with no such place the draw is from p."""
    V = 9001
    g, target, _ = _logits(B, B, 1, V, 0.0)
    dl = target.view(B, 2, -1)[:, 0].clone()
    for b in range(B):
        if b % 5:
            at = torch.randint(1, V, (b % 5 * 3,), generator=g)
            dl[b, at] = torch.nextafter(dl[b, at], torch.full_like(dl[b, at], 50.0 * (-1) ** b))
    draft, u = torch.zeros(B, 1, dtype=torch.int32), torch.full((B, 1), 2.0)      # u outside [0, 1): always refused
    noise = torch.empty(B, target.shape[1]).exponential_(generator=g).clamp_(min=1e-30)
    _same(target, dl, draft, u, noise, V, 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [50, 9001])
@pytest.mark.parametrize("B", [4, 90])
def test_residuals_that_fp32_does_not_hold(B, V):
    """All of p and of q but e^-100 lies on one token, so that the residual is among weights that fp32 has none of."""
    g = torch.Generator().manual_seed(B + V)
    ld = (V + 3) // 4 * 4
    target = -100 - 20 * torch.rand(B * 2, ld, generator=g)
    dl = -100 - 20 * torch.rand(B, ld, generator=g)
    top = torch.randint(0, V, (B,), generator=g)
    rows = target.view(B, 2, ld)[:, 0]
    at = torch.arange(B)
    rows[at, top] = 0.0
    dl[at, top] = 0.0
    draft = (dl[:, :V] - rows[:, :V]).argmax(1, keepdim=True).int()      # q(x) far above p(x): refused
    u = torch.full((B, 1), 0.99)
    noise = torch.empty(B, ld).exponential_(generator=g).clamp_(min=1e-30)
    p, q = _probs64(rows[:, :V], 1.0), _probs64(dl[:, :V], 1.0)
    assert (p[at, top] == 1).all() and (q[at, top] == 1).all()
    assert not np.isin(verify(target, dl, draft, [1] * B, u, noise, V, 1.0)[0][:, 0], top.numpy()[:, None]).all()
    _same(target, dl, draft, u, noise, V, 1.0)
