"""examples/decoder_layer.py: every call of a layer step against the oracle, on that call's own
inputs, eagerly and from a graph."""
import importlib.util
import os

import numpy as np
import pytest

import dense_gemm_sm_gb300 as dg
import oracle
from oracle import serving as ref

from .helpers import host_bf16_bits, torch_mod

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    t = torch_mod()
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("decoder_layer", os.path.join(ROOT, "examples", "decoder_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def f32(t):
    return t.detach().float().cpu().numpy()


@pytest.mark.parametrize("batch,graphed", [(3, False), (3, True), (20, True)])
def test_layer_step(example, batch, graphed):
    torch = torch_mod()
    width, hq, hkv, d, experts, inter, top, page = 256, 8, 2, 64, 8, 136, 2, 16
    layer = example.DecoderLayer(batch, width, hq, hkv, d, experts, inter, top, page, max_tokens=64)
    rng = np.random.default_rng(3)
    pool = ref.Kv4Pool(layer.pool.shape[0], page, hkv, d)
    k, v = (ref.bf16(rng.standard_normal((batch, 21, hkv * d))) for _ in range(2))

    def dev(x):
        return torch.from_numpy(ref.bf16_bits(x).view(np.int16)).view(torch.bfloat16).cuda()

    layer.prompt(dev(k), dev(v))
    layer.grow(8)
    table = layer.table.cpu().numpy()
    at = np.arange(21)
    for b in range(batch):
        pool.append(k[b].reshape(21, hkv, d), v[b].reshape(21, hkv, d), table[b, at // page] * page + at % page)
    layer.x.copy_(dev(ref.bf16(rng.standard_normal((batch, width)))))
    if graphed:
        keep = (layer.pool.clone(), layer.h.clone())
        layer.advance()
        graph = layer.capture()
        layer.pool.copy_(keep[0])
        layer.h.copy_(keep[1])
        layer.lens.sub_(1)
    scale = float(np.float32(1 / np.sqrt(d)))
    for _ in range(2):
        x, h0 = f32(layer.x), f32(layer.h)
        layer.advance()
        if graphed:
            graph.replay()
        else:
            layer.step()
        torch.cuda.synchronize()
        assert dg.dg_device_status() == dg.DG_OK
        rel = (width / 32 + 40) * 2.0 ** -25 + 8 * ref.F32
        # norm to codes, on x and h
        h1, y = ref.rmsnorm(x, h0, np.ones(width, np.float32), example.EPS)
        want, s = ref.rmsnorm_codes(y)
        a = layer.a.view(torch.float8_e4m3fn).float().cpu().numpy()
        assert np.all(np.abs(a - want) <= np.abs(want) * (ref.E4M3 + 4 * rel) + 2.0 ** -10)
        assert np.all(np.abs(layer.a_scale.cpu().numpy() - s) <= s * 4 * rel)
        # the projection, on the codes that it read
        n = (hq + 2 * hkv) * d
        C, D = oracle.gemm_fp8(batch, n, width, layer.a.cpu().numpy(), width, layer.a_scale.cpu().numpy(),
                               layer.wqkv.cpu().numpy(), width, layer.wqkv_scale.cpu().numpy())
        assert oracle.check_bf16(host_bf16_bits(layer.qkv), C, D)[0]
        # the cache, bit for bit on that projection's keys and values
        qkv = f32(layer.qkv)
        slots = layer.slots.cpu().numpy()
        pool.append(qkv[:, hq * d:(hq + hkv) * d].reshape(batch, hkv, d), qkv[:, (hq + hkv) * d:].reshape(batch, hkv, d), slots)
        assert np.array_equal(layer.pool.cpu().numpy(), pool.pack())
        # attention over it
        q = qkv[:, :hq * d].reshape(batch, 1, hq, d).astype(np.float64)
        want, bound = ref.kv4_attention(pool, q, layer.table.cpu().numpy(), layer.lens.cpu().numpy(), scale)
        got = f32(layer.attn).reshape(want.shape)
        assert np.all(np.abs(got - want) <= bound)
        # the output projection, the second norm, the router, the experts
        C, D = oracle.gemm(batch, width, hq * d, 1.0, host_bf16_bits(layer.attn), hq * d, host_bf16_bits(layer.wo), width, absden=True)
        assert oracle.check_bf16(host_bf16_bits(layer.o), C[0], D[0])[0]
        h2, y = ref.rmsnorm(f32(layer.o), h1.astype(np.float32), np.ones(width, np.float32), example.EPS)
        assert np.all(np.abs(f32(layer.h) - h2) <= 4 * ref.F32 * (np.abs(h1) + np.abs(h2)))
        assert np.all(np.abs(f32(layer.y) - y) <= np.abs(y) * (ref.BF16 + 2 * rel) + 4 * ref.F32 * np.abs(h1).max() * np.abs(y).max())
        C, D = oracle.gemm(batch, experts, width, 1.0, host_bf16_bits(layer.y), width, host_bf16_bits(layer.wr), experts, absden=True)
        assert oracle.check_f32(f32(layer.logits), C[0], D[0])[0]
        want, bound = ref.moe(f32(layer.y), f32(layer.logits), f32(layer.wg), f32(layer.wu), f32(layer.wd), top, True)
        assert np.all(np.abs(f32(layer.out) - want) <= bound)
        layer.x.copy_(layer.out)
