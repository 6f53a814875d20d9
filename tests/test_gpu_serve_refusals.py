"""Refusals of the W8A8 layer and the KV cache with tensors on the device (needs an MI355X): the short path of a call hands
everything that is not well-formed on to the full checks, which name the problem in an AtomError.  No call here launches."""
import pytest

torch = pytest.importorskip("torch")
import bit_quantized_gemm_amd as bq  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm GPU visible")
    bq.load_library()


def z(*shape, dtype=torch.float16, device="cuda"):
    return torch.zeros(shape, dtype=dtype, device=device)


def i32(*shape, **k):
    return z(*shape, dtype=torch.int32, **k)


def slots(*shape, dtype=torch.int64, **k):
    return z(*shape, dtype=dtype, **k)


@pytest.mark.parametrize("bad", [lambda: slots(), lambda: slots(5, 1), lambda: slots(4), lambda: slots(10)[::2], lambda: slots(5).int(),
                                 lambda: slots(5, device="cpu"), lambda: slots(0), lambda: [0] * 5])
def test_slots(bad):
    cache, K = bq.kv4_cache(3, 16, 2, 64), z(5, 2, 64)
    with pytest.raises(bq.AtomError, match="slots|shape"):
        bq.atom_kv4_append(K, K, bad(), cache)
    if not (isinstance(s := bad(), torch.Tensor) and s.shape == (4,)):         # any number of slots may be read
        with pytest.raises(bq.AtomError):
            bq.atom_kv4_read(cache, s)


def test_append_and_read():
    cache, K, s = bq.kv4_cache(3, 16, 2, 64), z(5, 2, 64), slots(5)
    for call in (lambda: bq.atom_kv4_append(z(), K, s, cache), lambda: bq.atom_kv4_append(K, z(), s, cache),
                 lambda: bq.atom_kv4_append(K, K[:, :1], s, cache), lambda: bq.atom_kv4_append(K, K.bfloat16(), s, cache),
                 lambda: bq.atom_kv4_append(K, K.cpu(), s, cache), lambda: bq.atom_kv4_append(K, K, s, cache._replace(v=cache.k)),
                 lambda: bq.atom_kv4_append(K, K, s, cache._replace(k=z(), v=z())), lambda: bq.atom_kv4_append(K, K, s, None),
                 lambda: bq.atom_kv4_append(K, K, s, bq.KV4Cache(*(t.cpu() for t in cache))),
                 lambda: bq.atom_kv4_append(K, K, s, cache._replace(k_par=[0])),
                 lambda: bq.atom_kv4_append(z(5, 64, 2).transpose(1, 2), K, s, cache),
                 lambda: bq.atom_kv4_append(z(1, 2, 64).expand(5, 2, 64), K, s, cache),
                 lambda: bq.atom_kv4_read(cache, s, dtype=torch.float32), lambda: bq.atom_kv4_read(cache[:2], s),
                 lambda: bq.atom_kv4_read(cache, s, K=z(5, 2, 32)), lambda: bq.atom_kv4_read(cache, s, K=K, V=K)):
        with pytest.raises(bq.AtomError):
            call()


def test_attention():
    cache, Q, table, lens, start = bq.kv4_cache(3, 16, 2, 64), z(5, 4, 64), i32(2, 3), i32(2), i32(3)

    def call(**k):
        a = {**dict(Q=Q, cache=cache, table=table, lens=lens, q_start=start), **k}
        return lambda: bq.atom_kv4_attention(**a)
    for bad in (dict(Q=z()), dict(Q=z(5, 3, 64)), dict(Q=z(5, 4, 128)), dict(Q=z(0, 4, 64)), dict(Q=Q.float()), dict(Q=z(4, 5, 64).transpose(0, 1)),
                dict(table=i32()), dict(table=i32(6)), dict(table=i32(0, 3)), dict(table=i32(2, 0)), dict(table=table.long()),
                dict(table=i32(3, 2).t()), dict(lens=i32()), dict(lens=i32(3)), dict(lens=i32(2, device="cpu")),
                dict(q_start=i32()), dict(q_start=i32(2)), dict(q_start=start.long()), dict(out=z(5, 4, 32)), dict(out=z()),
                dict(out=z(5, 4, 64, dtype=torch.bfloat16)), dict(out=Q), dict(workspace=z(4, 4, dtype=torch.uint8)),
                dict(workspace=z(4)), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(cache=None),
                dict(cache=cache._replace(v_par=cache.k_par[:2]))):
        with pytest.raises(bq.AtomError):
            print(bad, flush=True)
            call(**bad)()


def test_linear():
    X, Wq, sw = z(4, 200), z(6, 256, dtype=torch.int8), z(6, dtype=torch.float32)
    for call in (lambda: bq.linear_w8a8(z(), Wq, sw), lambda: bq.linear_w8a8(X[0], Wq, sw), lambda: bq.linear_w8a8(z(0, 200), Wq, sw),
                 lambda: bq.linear_w8a8(z(4, 0), Wq, sw), lambda: bq.linear_w8a8(X, Wq[:, :200], sw), lambda: bq.linear_w8a8(X, Wq[0], sw),
                 lambda: bq.linear_w8a8(X, Wq, sw[:5]), lambda: bq.linear_w8a8(X, Wq, z()), lambda: bq.linear_w8a8(X, Wq, sw, bias=z()),
                 lambda: bq.linear_w8a8(X, Wq, sw, bias=z(6).bfloat16()), lambda: bq.linear_w8a8(X.float(), Wq, sw),
                 lambda: bq.linear_w8a8(X, Wq.cpu(), sw), lambda: bq.linear_w8a8(X[:1].expand(4, 200), Wq, sw),
                 lambda: bq.linear_w8a8(z(200, 4).t(), Wq, sw), lambda: bq.linear_w8a8(X, Wq, sw, Y=z(4, 5)),
                 lambda: bq.linear_w8a8(X, Wq, sw, Y=z()), lambda: bq.linear_w8a8(X, Wq, sw, workspace=z())):
        with pytest.raises(bq.AtomError):
            call()
