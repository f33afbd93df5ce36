// Prints the restoring rule's choices: reads "m out con" lines, writes "fits pays decodes".
#include <stdio.h>

#include "dense_rule.h"

int main() {
  long long m, out, con;
  while (scanf("%lld %lld %lld", &m, &out, &con) == 3)
    printf("%d %d %d\n", qlora::dense_fits(m, out, con) ? 1 : 0, qlora::dense_pays(m, out, con) ? 1 : 0,
           qlora::gated_decodes(m, out, con) ? 1 : 0);
}
