"""AdamW's random rounding: which numbers a tensor gets, and the hardware's
conversion against its definition."""

import numpy as np
import pytest
import torch

import blockwise_scaled_fp8_amd as fp8
from oracle import e4m3, train
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


def _twins(gpu, count, n=4096):
    """Equal parameters with equal gradients."""
    g = torch.Generator().manual_seed(3)
    p, d = torch.randn(n, generator=g).bfloat16(), torch.randn(n, generator=g).bfloat16()
    out = []
    for _ in range(count):
        q = torch.nn.Parameter(p.to(gpu))
        q.grad = d.to(gpu)
        out.append(q)
    return out


def _codes(opt, p):
    return [opt.state[p][k] for k in ("exp_avg", "exp_avg_root")]


def test_groups_round_apart(gpu):
    """Equal tensors in different groups, as with and without decay, get random
    numbers of their own."""
    ps = _twins(gpu, 4)
    opt = fp8.AdamW([{"params": ps[:2]}, {"params": ps[2:], "weight_decay": 0.0}], state_bits=8)
    say("adamw groups")
    opt.step()
    for i in range(4):
        for j in range(i):
            for a, b in zip(_codes(opt, ps[i]), _codes(opt, ps[j])):
                # neighbouring codes where both remainders and random numbers allow: about
                # a third of the elements differ; independent halves never agree throughout
                assert float((a != b).float().mean()) > 0.1, (i, j)


def test_one_group_keeps_its_numbers(gpu):
    """All tensors in one group round as one call over them does."""
    ps, raw = _twins(gpu, 3), _twins(gpu, 3)
    opt = fp8.AdamW(ps, lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1, state_bits=8, seed=5)
    n = raw[0].numel()
    m, r = ([torch.zeros(n, dtype=torch.uint8, device=gpu) for _ in raw] for _ in range(2))
    ms, rs = ([torch.ones(n // 128, device=gpu) for _ in raw] for _ in range(2))
    say("adamw one group")
    opt.step()
    fp8.adamw_step([p.detach() for p in raw], [p.grad for p in raw], m, r, step=1, lr=1e-2, beta1=0.9, beta2=0.95,
                   eps=1e-8, weight_decay=0.1, exp_avg_scales=ms, root_scales=rs, seed=5 + 0x9E3779B97F4A7C15)
    for i in range(3):
        assert torch.equal(ps[i], raw[i])
        assert all(torch.equal(a, b) for a, b in zip(_codes(opt, ps[i]), (m[i], r[i])))


def test_neighbours_without_gradients_change_nothing(gpu):
    """A tensor's random numbers do not hang on which others have gradients, or
    on the step at which the others began."""
    full, part = _twins(gpu, 5), _twins(gpu, 5)
    a = fp8.AdamW([{"params": full[:3]}, {"params": full[3:]}], state_bits=8)
    b = fp8.AdamW([{"params": part[:3]}, {"params": part[3:]}], state_bits=8)
    part[0].grad = part[3].grad = None
    say("adamw missing gradients")
    a.step()
    b.step()
    for i in (1, 2, 4):
        assert torch.equal(full[i], part[i])
        assert all(torch.equal(x, y) for x, y in zip(_codes(a, full[i]), _codes(b, part[i])))
    # at its own second step a tensor rounds as it does beside tensors at theirs
    part[0].grad = full[0].grad
    b.step()
    a.step()
    for i in (1, 2, 4):
        assert torch.equal(full[i], part[i])


def test_ordinals(gpu):
    """adamw_step's ordinals pick the random numbers; without them the places
    in the lists do."""
    def state(n):
        z = [torch.zeros(n, dtype=torch.uint8, device=gpu) for _ in range(2)]
        s = [torch.ones(-(-n // 128), device=gpu) for _ in range(2)]
        return z + s
    n = 1000
    say("adamw ordinals")
    g = torch.randn(n, generator=torch.Generator().manual_seed(1)).to(gpu)
    results = {}
    for name, ordinals, place in (("seventh", [7], 0), ("list", None, 7), ("first", None, 0), ("last", [1000], 0)):
        count = place + 1
        p = [torch.zeros(n, device=gpu) for _ in range(count)]
        st = [state(n) for _ in range(count)]
        fp8.adamw_step(p, [g] * count, [s[0] for s in st], [s[1] for s in st], exp_avg_scales=[s[2] for s in st],
                       root_scales=[s[3] for s in st], step=1, lr=0.1, seed=9, ordinals=ordinals)
        results[name] = st[place]
    assert all(torch.equal(a, b) for a, b in zip(results["seventh"], results["list"]))
    assert not torch.equal(results["seventh"][0], results["first"][0])
    assert not torch.equal(results["seventh"][0], results["last"][0])
    p, s = torch.zeros(n, device=gpu), state(n)
    for bad in ([0, 1], [-1], [1 << 31]):
        with pytest.raises(ValueError):
            fp8.adamw_step([p], [g], [s[0]], [s[1]], exp_avg_scales=[s[2]], root_scales=[s[3]], step=1, lr=0.1, seed=9,
                           ordinals=bad)
    with pytest.raises(ValueError):
        fp8.adamw_step([p, p], [g, g], [s[0]] * 2, [s[1]] * 2, exp_avg_scales=[s[2]] * 2, root_scales=[s[3]] * 2, step=1,
                       lr=0.1, seed=9, ordinals=[4, 4])


def test_random_conversion_is_its_definition(gpu):
    """A million values over 22 octaves: with beta1 = 0 and beta2 = 0 the codes
    are those of the gradient and its magnitude, up or down by the remainder
    plus 16 random bits exactly."""
    n = 1 << 20
    g = torch.Generator().manual_seed(8)
    value = (torch.randn(n, generator=g) * torch.exp2(torch.rand(n, generator=g) * 22 - 17)).clamp(-440, 440)
    value[::128] = 448.0 * torch.where(torch.arange(n // 128) % 2 == 0, 1.0, -1.0)   # every block's scale is 1
    z = [torch.zeros(n, dtype=torch.uint8, device=gpu) for _ in range(2)]
    s = [torch.ones(n // 128, device=gpu) for _ in range(2)]
    say("adamw conversion")
    fp8.adamw_step([torch.zeros(n, device=gpu)], [value.to(gpu)], [z[0]], [z[1]], exp_avg_scales=[s[0]], root_scales=[s[1]],
                   step=1, lr=0.0, beta1=0.0, beta2=0.0, seed=12345)
    assert bool((s[0] == 1).all())
    bits = train.random_bits(12345, 0, n)[0]
    want = train.e4m3_stochastic(value.double().numpy(), bits)
    assert np.array_equal(e4m3.decode(z[0].cpu().numpy()), want)


def test_elements_past_32_bits_round_apart(gpu):
    """Element 2^32 + k does not get element k's random number."""
    k, n = 4096, (1 << 32) + 4096
    p, grad = (torch.zeros(n, dtype=torch.bfloat16, device=gpu) for _ in range(2))
    m, r = (torch.zeros(n, dtype=torch.uint8, device=gpu) for _ in range(2))
    s = [torch.ones(n // 128, device=gpu) for _ in range(2)]
    grad[:k] = torch.randn(k, generator=torch.Generator().manual_seed(1)).bfloat16().to(gpu)
    grad[-k:] = grad[:k]
    say("adamw past 2^32")
    fp8.adamw_step([p], [grad], [m], [r], exp_avg_scales=[s[0]], root_scales=[s[1]], step=1, lr=0.1, seed=9)
    alone = [t[:k].clone() for t in (m, r)]
    for t, a in zip((m, r), alone):
        assert float((t[-k:] != a).float().mean()) > 0.1
    assert torch.equal(s[0][:k // 128], s[0][-k // 128:]) and not m[k:-k].any()
