// Stand-ins for the launchers of the attention half, linked with its ABI file alone for the
// host sanitizer build: reaching one is an error.
#include <stdio.h>
#include <stdlib.h>

#include "qmoe_attn_internal.h"

namespace qmoe {

static hipError_t unexpected(const char* what) {
  fprintf(stderr, "launcher reached in the host-only build: %s\n", what);
  abort();
}

hipError_t launch_rows(const RowsArgs&) { return unexpected("launch_rows"); }
hipError_t launch_attn_decode(const AttnArgs&, const AttnPlan&) {
  return unexpected("launch_attn_decode");
}
hipError_t launch_attn_prefill(const AttnArgs&, const AttnPlan&) {
  return unexpected("launch_attn_prefill");
}

}  // namespace qmoe
