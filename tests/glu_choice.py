"""The library's choice of kernels for the gated layer and the 8-bit integer products, asked of its own rules: a
small program around csrc/gl_glu_choice.hpp, built by the host compiler (not collected by
pytest)."""
import os
import subprocess

import grouped_gemm_gl_amd as gl

CSRC = os.path.join(os.path.dirname(gl.__file__), "csrc")
IN = {"bf16": 0, "f32": 1, "f16": 2, "int8": 3}

SOURCE = r"""
#include <cstdio>
#include <cstring>
#include "gl_glu_choice.hpp"
int main() {
  char what[8];
  long long in, G, T, K, F, x;
  const char *form[] = {"full", "ragged", "ragged once", "written once"};
  while (scanf("%7s %lld %lld %lld %lld %lld %lld", what, &in, &G, &T, &K, &F, &x) == 7) {
    if (!strcmp(what, "glu")) {  // x: plain
      const gl::GluChoice c = gl::choose_glu((int)in, x != 0, G, T, K, F);
      if (c.kernel == gl::GluChoice::kFew) printf("few\n");
      else if (c.kernel == gl::GluChoice::kTile) printf("256 %s\n", form[c.ragged]);
      else printf("%dx%d%s%s\n", c.rows, c.weight_rows, c.parts == 2 ? " parts" : "", c.once ? " once" : "");
    } else {  // dx, dw, dw32 (fp32 gradients)
      const bool wgrad = what[1] == 'w';
      const gl::BackChoice c = gl::choose_glu_back((int)in, wgrad, !strcmp(what, "dw32"), G, T, K, 2 * F);
      if (c.rows == 256) printf("256 %s\n", form[c.tiles]);
      else printf("%dx%d%s%s\n", c.rows, c.cols, c.parts == 2 ? " parts" : "", c.once ? " once" : "");
    }
  }
}
"""


def build(folder):
    """The program's path."""
    src, exe = os.path.join(folder, "choice.cpp"), os.path.join(folder, "choice")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-o", exe, src], check=True, timeout=120)
    return exe


def ask(exe, questions):
    """Labels of (what, type, G, T, K, F, plain), what being glu, dx, dw or dw32 (fp32 gradients)."""
    lines = "".join(f"{w} {IN[t]} {G} {T} {K} {F} {int(p)}\n" for w, t, G, T, K, F, p in questions)
    out = subprocess.run([exe], input=lines, stdout=subprocess.PIPE, text=True, check=True, timeout=60).stdout.splitlines()
    assert len(out) == len(questions)
    return out
