"""The attention half of a layer as it is used -- q|k|v projection, adapters, rotation and append,
attention, o projection, adapters -- over several steps, eagerly and replayed as a graph: every
stage against its plain form on the stage's own input."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantised_decode_mat_gb300 as q  # noqa: E402
from quantised_decode_mat_gb300 import step as S  # noqa: E402
from tests import kv_plain as P  # noqa: E402

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]
DEV = "cuda"


def adapters(n, rank, K, rows, seed):
    g = torch.Generator().manual_seed(seed)
    return S.Adapters((torch.randn((n, rank, K), generator=g) / K ** 0.5).half().to(DEV),
                      torch.randn((n, rows, rank), generator=g).half().to(DEV), (torch.rand(n, generator=g) + 0.5).to(DEV))


def bits(t):
    return t.contiguous().view(torch.int32)


def host(cache):
    return P.Cache(*[t.cpu().numpy().copy() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)])


@pytest.mark.parametrize("rows_each,heads,kv_heads,head_dim", [([1, 1, 1], 16, 4, 64), ([4, 1, 2], 8, 2, 128)])
def test_steps_of_a_block(rows_each, heads, kv_heads, head_dim):
    from quantised_decode_mat_gb300 import build as qbuild
    qbuild.build()
    seqs, rows, hidden = len(rows_each), sum(rows_each), 1024
    block, table = S.make_attention_block(rows, seqs, 200, heads, kv_heads, head_dim, hidden, page_tokens=32)
    width = (heads + 2 * kv_heads) * head_dim
    block.qkv_adapters = adapters(3, 8, hidden, width, 1)
    block.o_adapters = adapters(3, 16, heads * head_dim, hidden, 2)
    start = np.concatenate(([0], np.cumsum(rows_each))).astype(np.int32)
    kv_len = torch.tensor([0, 37, 100], dtype=torch.int32, device=DEV)
    step = torch.tensor(rows_each, dtype=torch.int32, device=DEV)
    batch = q.KVBatch(table, kv_len, torch.from_numpy(start).to(DEV), max(rows_each), rows)
    adapter = torch.tensor([(i % 4) - 1 for i in range(rows)], dtype=torch.int32, device=DEV)
    x = torch.zeros((rows, hidden), device=DEV)
    g = torch.Generator(device=DEV).manual_seed(5)
    rng = np.random.default_rng(0)
    # what the sequences already hold
    for codes, scale in ((block.cache.k, block.cache.k_scale), (block.cache.v, block.cache.v_scale)):
        codes.copy_(torch.from_numpy(rng.integers(-127, 128, tuple(codes.shape)).astype(np.int8)))
        scale.fill_(0.02)
    graph = None
    for n in range(7):
        x.copy_(torch.randn(x.shape, device=DEV, generator=g))
        kv_len.add_(step)
        before = host(block.cache)
        if n < 3:
            block.run(x, batch, adapter)
        else:
            if graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    block.run(x, batch, adapter)
            graph.replay()
        q.get_device_error()
        # the projections and the adapters beside them
        shared = q.qmatvec_x(q.Q4_K, block.W_qkv, None, x)
        a = block.qkv_adapters
        ref, bound = P.adapters(x.cpu().numpy(), shared.cpu().numpy(), a.A.cpu().double().numpy(), a.B.cpu().double().numpy(),
                                adapter.tolist(), a.scale.cpu().double().numpy())
        kv = block.qkv[:, block.q_width:].cpu().numpy()
        assert (np.abs(kv - ref[:, block.q_width:]) <= bound[:, block.q_width:]).all()
        # rotation and append, bit for bit from the same projection
        lens = kv_len.cpu().numpy()
        again = q.lora_add(x, shared, a.A, a.B, adapter, a.scale).cpu().numpy()
        assert np.array_equal(again[:, block.q_width:], kv)
        rope = block.rope.cpu().numpy()
        q_rot = P.append(before, table.cpu().numpy(), lens, start, kv[:, :block.kv_width].reshape(rows, kv_heads, head_dim),
                         kv[:, block.kv_width:].reshape(rows, kv_heads, head_dim), rope,
                         again[:, :block.q_width].reshape(rows, heads, head_dim), head_dim, True)
        assert np.array_equal(block.q.cpu().numpy().reshape(q_rot.shape).view(np.uint32), q_rot.view(np.uint32))
        now = host(block.cache)
        assert np.array_equal(now.k, before.k) and np.array_equal(now.v, before.v)
        assert np.array_equal(now.ks, before.ks) and np.array_equal(now.vs, before.vs)
        # attention, and the o projection of what it gave
        ref, bound = P.attention(now, table.cpu().numpy(), lens, start, q_rot, head_dim ** -0.5)
        assert (np.abs(block.attended.cpu().numpy().reshape(ref.shape) - ref) <= bound).all()
        o, b = q.qmatvec_x(q.Q4_K, block.W_o, None, block.attended), block.o_adapters
        assert torch.equal(bits(q.lora_add(block.attended, o, b.A, b.B, adapter, b.scale)), bits(block.y))
