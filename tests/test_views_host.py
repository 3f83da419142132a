"""views_overlap (csrc/api_util.cuh) against all elements of small random views, and on the layouts of q and k."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "api_util.cuh"
#include <cstdio>
int main() {
  qnre_tensor4_t t[2] = {};
  long long base[2], v[2][8];
  while (true) {
    for (int k = 0; k < 2; ++k) {
      if (std::scanf("%lld", &base[k]) != 1) return 0;
      for (int i = 0; i < 8; ++i)
        if (std::scanf("%lld", &v[k][i]) != 1) return 1;
      t[k].data = reinterpret_cast<void*>((1ll << 32) + 2 * base[k]);
      t[k].dtype = QNRE_DTYPE_BF16;
      for (int i = 0; i < 4; ++i) t[k].shape[i] = v[k][i], t[k].stride[i] = v[k][4 + i];
    }
    qnre::api::ByteRange r[2];
    if (qnre::api::check_view(&t[0], &r[0]) || qnre::api::check_view(&t[1], &r[1])) return 2;
    std::printf("%d\n", qnre::api::views_overlap(&t[0], r[0], &t[1], r[1]));
  }
}
"""


@pytest.fixture(scope="module")
def overlap(tmp_path_factory):
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    if shutil.which("g++") is None or not os.path.exists(os.path.join(cuda, "include", "cuda_runtime.h")):
        pytest.skip("no host compiler or CUDA headers")
    d = tmp_path_factory.mktemp("views")
    (d / "views.cpp").write_text(PROGRAM)
    exe = str(d / "views")
    subprocess.run(["g++", "-std=c++17", "-O1", "-w", f"-I{ROOT}/ulysses_qkv_proj_gb300/csrc", f"-I{ROOT}/include",
                    f"-I{cuda}/include", str(d / "views.cpp"), "-o", exe], check=True)

    def run(pairs):
        text = "\n".join(" ".join(map(str, [*v])) for pair in pairs for v in ([b, *shape, *stride] for b, shape, stride in pair))
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
        return [x == "1" for x in out.split()]
    return run


def elements(base, shape, stride):
    r = {base}
    for n, s in zip(shape, stride):
        r = {x + i * s for x in r for i in range(n)}
    return r


def test_against_all_elements(overlap):
    rng = random.Random(0)
    pairs = []
    for _ in range(4000):
        D = rng.choice([1, 2, 4])
        if rng.random() < 0.7:      # bands of one buffer: the same strides, in any order of the axes
            order = rng.sample(range(3), 3)
            ext = [rng.randint(1, 4) for _ in range(3)]
            stride, at = [0] * 3, D
            for i in order:
                stride[i] = at
                at *= ext[i] + rng.randint(0, 2)
            views = []
            for _ in range(2):
                shape = [rng.randint(1, e) for e in ext]
                base = sum(rng.randint(0, e - n) * s for e, n, s in zip(ext, shape, stride)) + rng.choice([0, 0, 0, rng.randint(0, D)])
                views.append((base, [*shape, D], [*stride, 1]))
        else:
            views = [(rng.randint(0, 60), [rng.randint(1, 4) for _ in range(3)] + [D], [rng.randint(1, 40) for _ in range(3)] + [1])
                     for _ in range(2)]
        pairs.append(views)
    want = [not elements(*a).isdisjoint(elements(*b)) for a, b in pairs]
    assert overlap(pairs) == want
    assert 500 < sum(want) < 3500


def test_bands_of_one_buffer(overlap):
    """q, k and v heads of a buffer [B, S, H, D], [B, H, S, D] or [S, B, H, D]: apart, unless a head is in both."""
    B, S, H, D, Hq, Hk = 3, 1000, 72, 128, 56, 8
    for st in ([S * H * D, H * D, D, 1], [S * H * D, D, S * D, 1], [H * D, B * H * D, D, 1]):
        band = lambda h, n: (h * st[2], [B, S, n, D], st)
        assert overlap([(band(0, Hq), band(Hq, Hk)), (band(Hq, Hk), band(0, Hq)), (band(Hq, Hk), band(Hq + Hk, Hk)),
                        (band(0, Hq), band(Hq - 1, Hk)), (band(Hq, Hk), band(Hq + Hk - 1, 1)), (band(0, 1), band(1, 1)),
                        (band(3, 1), band(3, 1))]) == [False, False, False, True, True, False, True]
        # a token further on
        q, k = band(0, Hq), band(Hq, Hk)
        assert overlap([(q, (st[1], [B, S - 1, Hq, D], st)), (q, (k[0] + st[1], [B, S - 1, Hk, D], st))]) == [True, False]


def test_strides_that_do_not_nest_are_taken_to_meet(overlap):
    assert overlap([((0, [5000, 5000, 1, 1], [2, 4, 1, 1]), (1, [5000, 5000, 1, 1], [4, 2, 1, 1]))]) == [True]
