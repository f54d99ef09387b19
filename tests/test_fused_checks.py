"""What the fused operators' checks reject, without a GPU: a right result passes
and results with one planted mistake do not."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from fused_ref import DT, w4_norm_close, w4_weights  # noqa: E402


@pytest.mark.parametrize("typ", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K,group", [(5, 40, 16384, 32), (16, 33, 17000, 64), (3, 100, 9001, 32),
                                         (64, 64, 4100, 96)])
def test_w4_norm_rejects_small_mistakes(M, N, K, group, typ):
    dt = DT[typ]
    r = torch.Generator().manual_seed(M + K)
    groups = -(-K // group)
    X = torch.randn((M, K), generator=r).to(dt)
    Wq = torch.randint(0, 256, (N, (K + 1) // 2), generator=r, dtype=torch.uint8)
    s = (torch.rand((N, groups), generator=r) + 0.5).to(dt)
    z = torch.randint(0, 16, (N, groups), generator=r, dtype=torch.uint8)
    q, sc = w4_weights(Wq, s, z, group, K)

    def product(x, q, sc):
        return (x.double() @ (q * sc).T).to(dt)

    w4_norm_close(product(X, q, sc), X, q, sc, "the definition")
    # fp32 sums of the bf16 form's two products, block by block of 128
    tot = torch.zeros((M, N))
    zz = z.float()[:, torch.arange(K) // group] + 128
    for k in range(0, K, 32):
        x, at = X[:, k:k + 32].float(), slice(k, k + 32)
        qz = (q[:, at].float() + zz[:, at])
        tot += (x @ qz.T - x.sum(1, keepdim=True) * zz[:, k]) * sc[:, k].float()
    w4_norm_close(tot.to(dt), X, q, sc, "two sums in fp32")

    def wrong(what, x=X, q=q, sc=sc):
        with pytest.raises(AssertionError):
            w4_norm_close(product(x, q, sc), X, *w4_weights(Wq, s, z, group, K), what)

    for last in (8, 16, 32):
        x = X.clone()
        x[:, -last:] = 0
        wrong("the last %d of K left out" % last, x=x)
    x = X.clone()
    x[:, 1024:1056] = 0
    wrong("a step of 32 left out", x=x)
    last = torch.arange(K) // group == groups - 1
    if groups > 1 and int(last.sum()) >= 8:
        sc2 = sc.clone()
        sc2[:, last] = s[:, groups - 2].double()[:, None]
        wrong("the last group's scale", sc=sc2)
        q2 = q.clone()
        q2[:, last] += 3
        wrong("the last group's zero point", q=q2)
    swapped = q.clone()
    swapped[:, 0:32:2], swapped[:, 1:32:2] = q[:, 1:32:2], q[:, 0:32:2]
    wrong("the nibbles of 16 bytes swapped", q=swapped)
