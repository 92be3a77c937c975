"""GPU parity of AdamW over many tensors: 32-bit states bit for bit with the
one-tensor step, 8-bit states against float64 from the codes they hold."""

import numpy as np
import pytest
import torch

from oracle import bf16, fp8, optim

pytestmark = pytest.mark.gpu
HP = dict(lr=2e-3, betas=(0.9, 0.995), eps=1e-8, weight_decay=0.01)
HP32 = [float(np.float32(v)) for v in (2e-3, 0.9, 0.995, 1e-8, 0.01)]
SIZES = [1, 7, 255, 256, 257, 4095, 4096, 4097, 0, 70001, 300_000]


@pytest.fixture(scope="module")
def q():
    import bit_nf4_quantized_06_b200 as q
    return q


def _tensors(sizes, seed, offset=0):
    g = torch.Generator().manual_seed(seed)
    t = [torch.randn(n + offset, generator=g) * 0.02 for n in sizes]
    return [v.cuda()[offset:] for v in t], [v.cuda().bfloat16()[offset:] for v in t], g


def _grads(sizes, g, offset=0):
    return [(torch.randn(n + offset, generator=g) * 0.01).cuda()[offset:] for n in sizes]


@pytest.mark.parametrize("sizes,offset", [(SIZES, 0), (SIZES, 1), ([5], 0), ([300] * 600, 0)])
def test_32_bit_states_as_the_one_tensor_step(q, sizes, offset):
    masters, params, g = _tensors(sizes, 1, offset)
    ref = [(p.clone(), b.clone(), torch.zeros_like(p), torch.zeros_like(p)) for p, b in zip(masters, params)]
    group = q.AdamWGroup(masters, params=params)
    for t in range(1, 4):
        grads = _grads(sizes, g, offset)
        before = q.qlora_launch_count()
        q.qlora_adamw_multi(group, grads, t, **HP)
        assert q.qlora_launch_count() - before <= -(-len(sizes) // 470)
        for (p, b, m, v), gr in zip(ref, grads):
            if p.numel():
                q.qlora_adamw_step(p, gr, m, v, t, param=b, **HP)
    torch.cuda.synchronize()
    at = 0
    for p, b, (rp, rb, rm, rv) in zip(masters, params, ref):
        n = p.numel()
        assert torch.equal(p, rp) and torch.equal(b, rb)
        assert torch.equal(group.m[at:at + n], rm) and torch.equal(group.v[at:at + n], rv)
        at += -(-n // 256) * 256
    assert q.qlora_device_status() == (0, 0)


def _blocks(values, n):
    wide = np.zeros(-(-n // 256) * 256)
    wide[:n] = values
    return wide.reshape(-1, 256)


@pytest.mark.parametrize("sizes,offset,with_params", [(SIZES, 0, True), (SIZES, 1, True), ([9, 100_000], 0, False)])
def test_8_bit_states_against_float64(q, sizes, offset, with_params):
    masters, params, g = _tensors(sizes, 2, offset)
    group = q.AdamWGroup(masters, params=params if with_params else None, bits=8)
    starts = np.concatenate([[0], np.cumsum([-(-n // 256) * 256 for n in sizes])]).astype(int)

    def state(codes, scales, i):
        a, n = starts[i], sizes[i]
        c = fp8.decode(codes.view(torch.uint8)[a:a + n].cpu().numpy(), fp8.E4M3)
        s = scales[a // 256:a // 256 + -(-n // 256)].double().cpu().numpy()
        return c * np.repeat(s, 256)[:n], s, c

    for t in range(1, 5):
        grads = _grads(sizes, g, offset)
        for gr in grads:
            if gr.numel() > 200:
                gr[50:150] *= 1e-6               # values far below their block's largest
        old = [(p.double().cpu().numpy(), state(group.m, group.m_scales, i)[0], state(group.v, group.v_scales, i)[0])
               for i, p in enumerate(masters)]
        q.qlora_adamw_multi(group, grads, t, **HP)
        torch.cuda.synchronize()
        for i, (p, gr) in enumerate(zip(masters, grads)):
            n = sizes[i]
            if n == 0:
                continue
            po, m, r = old[i]
            rp, rm, rv = optim.adamw_step(po, gr.double().cpu().numpy(), m, r * r, t, *HP32)
            rr = np.sqrt(rv)
            got = p.double().cpu().numpy()
            # fp32 arithmetic on the same states: as for the one-tensor step, an absolute part
            # where m cancels to near zero
            assert np.allclose(got, rp, rtol=1e-6, atol=1e-5 * HP["lr"])
            if with_params:
                want = bf16.round_f32_to_bf16_bits(p.cpu().numpy())
                assert np.array_equal(params[i].cpu().view(torch.int16).numpy().view(np.uint16), want)
            # m's terms are at most |m| + |g|: eight roundings of those; the root's relative error is smaller
            noise_m = 8 * 2.0 ** -24 * (np.abs(m) + np.abs(gr.double().cpu().numpy()))
            for (value, scale, code), ref, noise in ((state(group.m, group.m_scales, i), rm, noise_m),
                                                     (state(group.v, group.v_scales, i), rr, 8 * 2.0 ** -24 * rr)):
                top = np.maximum(np.abs(_blocks(ref, n)).max(1), 2.0 ** -100) / 448
                slack = np.abs(_blocks(noise, n)).max(1) / 448 + 2.0 ** -22 * top
                assert np.all(np.abs(scale - top) <= slack)
                wide = np.repeat(top, 256)[:n]
                half = np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * wide) * (1 + 2.0 ** -3)
                floor = np.where(ref > 0, 2.0 ** -9 * wide, 0) if ref is rr else 0
                off = np.abs(value - ref)
                assert np.all((off <= half + noise + 1e-5 * np.abs(ref)) | (off <= floor))
                if ref is rr:
                    assert np.all(code[rr > 0] > 0)      # no root above zero is lost
    assert q.qlora_device_status() == (0, 0)


@pytest.mark.parametrize("bits", [8, 32])
def test_a_gradient_that_is_not_finite_spoils_its_own_value_only(q, bits):
    masters, _, g = _tensors([1000, 300], 3)
    clean = [p.clone() for p in masters]
    a, b = q.AdamWGroup(masters, bits=bits), q.AdamWGroup(clean, bits=bits)
    grads = _grads([1000, 300], g)
    bad = [v.clone() for v in grads]
    bad[0][10], bad[0][700], bad[1][299] = float("nan"), float("inf"), float("-inf")
    hit = [torch.zeros(n, dtype=torch.bool, device="cuda") for n in (1000, 300)]
    hit[0][[10, 700]] = True
    hit[1][299] = True
    for v, h in zip(grads, hit):
        v[h] = 0
    for t in (1, 2):
        q.qlora_adamw_multi(a, bad if t == 1 else grads, t, **HP)
        q.qlora_adamw_multi(b, grads, t, **HP)
        for p, c, h in zip(masters, clean, hit):
            assert torch.all(torch.isnan(p[h])) and torch.equal(p[~h], c[~h])


def test_zero_gradients_and_first_step(q):
    masters, _, _ = _tensors([513], 5)
    p0 = masters[0].clone()
    group = q.AdamWGroup(masters, bits=8)
    q.qlora_adamw_multi(group, [torch.zeros(513, device="cuda")], 1, **HP)
    assert torch.equal(masters[0], p0 * np.float32(1 - HP32[0] * HP32[4]))      # decay alone, no 0/0
    assert torch.all(group.m.float() == 0) and torch.all(group.v.float() == 0) and torch.all(torch.isfinite(group.m_scales))


def test_refusals_padding_and_streams(q):
    masters, params, g = _tensors([100, 300], 6)
    grads = _grads([100, 300], g)
    group = q.AdamWGroup(masters, params=params, bits=8)
    for bad in (grads[:1], [grads[1], grads[0]], [grads[0], grads[1].double()], [grads[0].cpu(), grads[1]],
                [grads[0], torch.randn(600, device="cuda")[::2]]):
        with pytest.raises(ValueError):
            q.qlora_adamw_multi(group, bad, 1)
    with pytest.raises(q.QloraError):
        q.qlora_adamw_multi(group, grads, 0)
    same = q.AdamWGroup([masters[0], masters[0]])
    with pytest.raises(q.QloraError):
        q.qlora_adamw_multi(same, [grads[0], grads[0]], 1)
    for kw in (dict(bits=16), dict(m=torch.zeros(5, device="cuda")), dict(m_scales=torch.zeros(3, device="cuda")),
               dict(params=params[:1])):
        with pytest.raises(ValueError):
            q.AdamWGroup(masters, **kw)
    twin = [p.clone() for p in masters]
    other = q.AdamWGroup(twin, bits=8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q.qlora_adamw_multi(other, grads, 1, stream=side)
    q.qlora_adamw_multi(group, grads, 1)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(twin, masters))
    moved = q.AdamWGroup([p.clone() for p in masters])
    moved.masters[0].data = moved.masters[0].clone()
    with pytest.raises(ValueError):
        q.qlora_adamw_multi(moved, grads, 1)
    # a state put in the place of the group's own (it would not be the one that is updated)
    for name, bits in (("m", 8), ("v_scales", 8), ("v", 32)):
        put = q.AdamWGroup([p.clone() for p in masters], bits=bits)
        setattr(put, name, getattr(put, name).clone())
        with pytest.raises(ValueError):
            q.qlora_adamw_multi(put, grads, 1)


@pytest.mark.parametrize("bits", [8, 32])
def test_captured_and_replayed(q, bits):
    masters, _, g = _tensors([5000, 33], 7)
    twin = [p.clone() for p in masters]
    a, b = q.AdamWGroup(masters, bits=bits), q.AdamWGroup(twin, bits=bits)
    grads = _grads([5000, 33], g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.qlora_adamw_multi(a, grads, 3, **HP)
    for _ in range(3):
        graph.replay()
        q.qlora_adamw_multi(b, grads, 3, **HP)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(masters, twin))
    assert torch.equal(a.m.view(torch.uint8), b.m.view(torch.uint8))
