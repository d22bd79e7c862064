"""How a C program sees that the header declares the layer operators. On the CPU."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_macro(tmp_path):
    src = tmp_path / "have.c"
    src.write_text('#include "mamba3.h"\n#if !defined(MAMBA3_LAYER_OPERATORS) || MAMBA3_LAYER_OPERATORS < 1\n#error missing\n#endif\n'
                   "int main(void) { return 0; }\n")
    subprocess.run(["gcc", "-Werror", "-I", os.path.join(ROOT, "include"), "-fsyntax-only", str(src)], check=True)
