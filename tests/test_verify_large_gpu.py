"""smd_verify_drafts from 2^23 target probabilities on, where a request's CTAs are as many as load the SMs most
evenly (below: as many as a cluster takes), against whole numbers and fractions: every output is equal."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import paged4 as opaged4
from paged_common import i32

pytestmark = pytest.mark.gpu


def ctas(R, V, sms):
    """A request's CTAs: the most of those with the largest share of SMs at work over the rounds."""
    share = {c: R * c / (-(-R * c // sms) * sms) for c in range(1, 9) if c == 1 or V > 4096 * (c - 1)}
    return max(c for c in share if share[c] == max(share.values()))


@pytest.mark.parametrize("C,V", [(1, 4000), (2, 7000), (3, 11000), (5, None), (6, None), (7, None), (8, None)])
@pytest.mark.parametrize("given,off", [(True, 0), (True, 1), (False, 3)])
def test_as_many_ctas_as_load_the_sms_evenly(cuda, C, V, given, off):
    """Requests of which C CTAs each fill the GPU once (8: four times), or of as many CTAs as a short row allows,
    in rows at 16 bytes or off them by 4 and 12. Drafts that stay, that are refused at each place, draws at both
    ends; some requests are compared."""
    import torch
    from sparse_mla_decode_gb300 import binding
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    G = 3
    if V is None:
        R = sms // (C if C < 8 else 2)
        V = -(-2 ** 23 // R) // 4 * 4 + 4
    else:
        R = (-(-2 ** 23 // V) + sms) // sms * sms  # rounds that any number of CTAs fills
    V += off
    assert R * V >= 2 ** 23 and ctas(R, V, sms) == C
    g = torch.Generator(device=cuda).manual_seed(C + off)

    def rows(n):
        """[R, n, V] float32, `off` elements from a multiple of 16 bytes."""
        flat = torch.empty(R * n * V + off, device=cuda)
        x = flat[off:].view(R, n, V)
        x.copy_(torch.softmax(2 * torch.randn(R, n, V, generator=g, device=cuda), -1))
        return x

    p = rows(G)
    q = rows(G - 1) if given else None
    tokens = p[:, :G - 1].argmax(-1).int()
    rng = np.random.default_rng(C)
    accept, sample = rng.random((R, G - 1)), rng.random(R)
    accept[0::4] = 0.0                     # both stay
    accept[1::4] = 1.0 if not given else 1e9  # the first is refused
    accept[2::4, 0] = 0.0
    accept[2::4, 1] = 1.0 if not given else 1e9
    sample[0], sample[-1] = 0.0, np.nextafter(np.float32(1), np.float32(0))
    tokens[3::8, 1] = V  # no second draft
    accept, sample = accept.astype(np.float32), sample.astype(np.float32)
    got = binding.verify_drafts(p, tokens, torch.from_numpy(accept).to(cuda), torch.from_numpy(sample).to(cuda), draft=q)
    again = binding.verify_drafts(p, tokens, torch.from_numpy(accept).to(cuda), torch.from_numpy(sample).to(cuda), draft=q)
    torch.cuda.synchronize()
    pick = np.unique(np.r_[0:4, R // 2, R - 2:R])
    at = i32(pick, cuda).long()
    want = opaged4.verify_drafts(p[at].cpu().numpy(), None if q is None else q[at].cpu().numpy(), tokens[at].cpu().numpy(),
                                 accept[pick], sample[pick])
    for name, a, b, c in zip(("tokens", "accepted", "rejected"), got, again, want):
        assert torch.equal(a, b), name
        assert np.array_equal(a.cpu().numpy()[pick].astype(np.int64), c), name
    assert want[1][:3].tolist() == [2, 0, 1]
    drawn = got[0].gather(1, got[1].long()[:, None])
    assert bool(((drawn >= 0) & (drawn < V)).all())
