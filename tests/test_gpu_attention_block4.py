"""AttentionBlock over a 4-bit cache that is kept short: projection, append with positions, attention, weights,
o projection, then eviction, over several steps, eagerly and replayed as a graph; every stage against its
plain form on the stage's own input."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantised_decode_mat_gb300 as q  # noqa: E402
from quantised_decode_mat_gb300 import step as S  # noqa: E402
from tests import kv4_plain as P  # noqa: E402

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]
DEV = "cuda"


def host(cache):
    return P.Cache(*[t.cpu().numpy().copy() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)])


@pytest.mark.parametrize("heads,kv_heads,head_dim", [(16, 4, 64), (8, 2, 128)])
def test_steps_of_a_block_kept_short(heads, kv_heads, head_dim):
    from quantised_decode_mat_gb300 import build as qbuild
    qbuild.build()
    seqs, hidden, keep, sinks, recent = 3, 512, 40, 2, 12
    block, table = S.make_attention_block(seqs, seqs, 96, heads, kv_heads, head_dim, hidden, page_tokens=16, kv_bits=4,
                                          weigh=True, positions=300)
    lens = torch.tensor([0, 39, 50], dtype=torch.int32, device=DEV)
    position = torch.tensor([-1, 70, 99], dtype=torch.int32, device=DEV)  # of the rows last appended
    batch = q.KVBatch(table, lens)
    rng = np.random.default_rng(0)
    for codes, scale in ((block.cache.k, block.cache.k_scale), (block.cache.v, block.cache.v_scale)):
        codes.copy_(torch.from_numpy(rng.integers(0, 256, tuple(codes.shape)).astype(np.uint8)))
        scale.fill_(0.05)
    block.weights.copy_(torch.from_numpy(rng.exponential(1, tuple(block.weights.shape)).astype(np.float32)))
    x = torch.zeros((seqs, hidden), device=DEV)
    after = torch.zeros(seqs, dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(5)
    tab, start = table.cpu().numpy(), np.arange(seqs + 1).astype(np.int32)

    def one():
        lens.add_(1)
        position.add_(1)
        block.run(x, batch, positions=position)

    def thin():
        block.evict(batch, keep, sinks, recent, after)
        lens.copy_(after)

    graphs = None
    for n in range(6):
        x.copy_(torch.randn(x.shape, device=DEV, generator=g))
        before, old_w = host(block.cache), block.weights.cpu().numpy().copy()
        if n == 3:  # from here on replayed
            torch.cuda.synchronize()
            graphs = []
            for f in (one, thin):
                graphs.append(torch.cuda.CUDAGraph())
                with torch.cuda.graph(graphs[-1]):
                    f()
        graphs[0].replay() if graphs else one()
        q.get_device_error()
        now, L = host(block.cache), lens.cpu().numpy()
        proj = q.qmatvec_x(q.Q4_K, block.W_qkv, None, x).cpu().numpy()
        kv = proj[:, block.q_width:]
        assert np.array_equal(block.qkv[:, block.q_width:].cpu().numpy(), kv)
        q_rot = P.append(before, tab, L, start, kv[:, :block.kv_width].reshape(seqs, kv_heads, head_dim),
                         kv[:, block.kv_width:].reshape(seqs, kv_heads, head_dim), block.rope.cpu().numpy(),
                         proj[:, :block.q_width].reshape(seqs, heads, head_dim), head_dim, True, position.cpu().numpy())
        assert np.array_equal(block.q.cpu().numpy().reshape(q_rot.shape), q_rot)
        for a, b in ((now.k, before.k), (now.v, before.v), (now.ks, before.ks), (now.vs, before.vs)):
            assert np.array_equal(a, b)
        ref, bound, lref, lbound = P.attention(now, tab, L, start, q_rot, head_dim ** -0.5)
        assert (np.abs(block.attended.cpu().numpy().reshape(ref.shape) - ref) <= bound).all()
        lse = block.lse.cpu().numpy()
        assert (np.abs(lse - lref) <= lbound).all()
        wref, wbound = P.weigh(now, tab, L, start, q_rot, head_dim ** -0.5, lse, old_w)
        new_w = block.weights.cpu().numpy()
        assert (np.abs(new_w - wref) <= wbound).all()
        assert torch.equal(q.qmatvec_x(q.Q4_K, block.W_o, None, block.attended), block.y)
        graphs[1].replay() if graphs else thin()
        q.get_device_error()
        want, _ = P.evict(now, tab, L, new_w, keep, sinks, recent)
        assert lens.tolist() == want.tolist()
        thinned = host(block.cache)
        assert np.array_equal(thinned.k, now.k) and np.array_equal(thinned.vs, now.vs)
        assert np.array_equal(block.weights.cpu().numpy(), new_w)
    assert lens.tolist() == [6, 40, 40] and position.tolist() == [5, 76, 105]
